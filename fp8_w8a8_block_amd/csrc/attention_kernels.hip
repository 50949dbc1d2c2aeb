// Attention over the paged FP8 cache for gfx950: ragged batches, causal, with
// an optional sliding window and sinks, and batches behind a shared prefix.
//
// For a query row q at position p of its request (one row per query head):
//   s_j = scale * k_scale * <q, dec(K_j)>,  out = v_scale * sum_j softmax(s)_j dec(V_j)
// over the visible j.  One pass over the keys keeps a base m near the running
// maximum, the sum l = sum exp(s_j - m) and O = sum exp(s_j - m) V_j, rescaled
// when m moves.
//
// Numbers.  E4M3 codes convert exactly to bf16 and to fp16 (4 significant
// bits, 2^-9 .. 448), queries are bf16, so <q, K_j> is a sum of exact products
// on the bf16 matrix instruction with fp32 accumulation, and nothing of the
// scores is rounded below fp32.  P = exp(s - m) goes to fp16, 11 bits to the
// bf16 output's 8; the base keeps a row's largest P at 2^10 .. 2^15, so that
// weights down to 2^-24 of the largest have them all (see moved_base).  O is fp32,
// and l sums the fp32 values.  exp(x) is exp2(x log2 e), the factor folded into
// the score scale.
//
// Layout.  S^T = K Q^T puts one query row in each lane column, so m, l and the
// rescaling of O^T = V^T P^T stay in the lane's own column, and P's registers
// are the second product's operand as they are: the matrix instruction sums
// over its k index in any order, so the keys of a lane's P values (rows of the
// S^T tile it holds) are simply the keys whose V bytes it is given.
//
// Rows.  The G = Hq / Hk query heads of a KV head share its keys: row rho of
// request r and KV head h is token rho / G, head h G + rho % G.
//
// Work.  An item is (request, row tile, KV head); its cost is the number of
// key tiles its mask leaves.  A fixed grid of workgroups takes even shares of
// the whole list's tiles, found by a prefix sum over the requests that every
// workgroup forms itself, so no length is needed on the host and ragged
// batches, one long context and many short ones all fill the card.  Items of a
// few tiles, a prompt's first ones, take longer than their tiles say: their start
// and end are not counted.  An item inside one share is finished there; one that
// shares cut leaves fp32 partial rows (O, m, l) in the workspace, and a second
// launch joins them.
#include <atomic>

#include "attention_launch.h"
#include "device_common.h"
#include "launch.h"

namespace fp8k {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
#define FP8_NEG_INF (-__builtin_inff())

// ---- workspace -----------------------------------------------------------------
// descriptor of an item that starts in a workgroup's share and ends in a later one
struct Split {
  int32_t token0;      // the request's first token
  int32_t row0, rows;  // rows of the tile
  int32_t head;        // KV head
  int32_t parts;       // workgroups that hold a part of it (0: none starts here)
  int32_t pad[3];
};

// partial rows of a launch: workgroup w writes slot 2 w (an item that began
// before its share) and slot 2 w + 1 (one that goes on behind it)
struct Parts {
  float* ml;           // [slots][R][2]: base m (of the scores times log2 e) and l
  float* o;            // [slots][R][D]
  Split* split;        // [workgroups]
  // shared prefix only: where each row's result is, and rows that one
  // workgroup finished
  int2* where;         // [T * Hq]: row of ml / o of the first part, number of parts
                       // (0: in whole_*; < 0: a row of no request)
  int2* reset;         // where[] of the launch behind this one, set to "of no request"
  float* whole_ml;     // [T * Hq][2]
  float* whole_o;      // [T * Hq][D]
};

// ---- division -------------------------------------------------------------------
// x / d for x < 2^51, inv = 1 / d: (x + 1/2) / d lies at least 1 / (2 d) from a
// whole number, the fp64 error is below x / d * 2^-51.
__device__ __forceinline__ uint32_t div32(uint32_t x, double inv) {
  return (uint32_t)__builtin_fma((double)x, inv, 0.5 * inv);
}
__device__ __forceinline__ int64_t div64(int64_t x, double inv) {
  return (int64_t)__builtin_fma((double)x, inv, 0.5 * inv);
}

// ---- which keys a row tile needs ------------------------------------------------
struct Request {
  int token0, n;       // first query token, query tokens
  int p0;              // position of the first one
  int keys;            // keys that the table can hold and the length names
};

// keys of a request: key indices of the tiles that are read ahead of its last one,
// at most 6 of 128 keys, stay below 2^31
constexpr int kMostKeys = 0x7fff0000;
__device__ __forceinline__ int keys_of(const AttentionArgs& a, int len, int32_t width) {
  int64_t cap = a.num_blocks > 0 ? (int64_t)width * a.page : 0;
  cap = cap < kMostKeys ? cap : kMostKeys;
  return len < 0 ? 0 : (int64_t)len < cap ? len : (int)cap;
}

struct Tiles {
  int sink;            // tiles 0 .. sink - 1, then
  int first, last;     // tiles first .. last - 1
  int p_lo, p_hi;      // positions of the tile's first and last token
  __device__ __forceinline__ int count() const { return sink + last - first; }
  __device__ __forceinline__ int key_tile(int k) const { return k < sink ? k : first + k - sink; }
};

// kPrefix: the rows are all T tokens and see all of the prefix.
template <bool kPrefix>
__device__ __forceinline__ Request load_request(const AttentionArgs& a, int r) {
  Request q;
  if (kPrefix) {
    q.token0 = 0;
    q.n = a.T;
    q.keys = keys_of(a, a.prefix_len[0], a.prefix_width);
    q.p0 = q.keys - 1;
  } else {
    int lo = a.offsets[r], hi = a.offsets[r + 1];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    const int len = a.lens[r] > 0 ? a.lens[r] : 0;
    q.token0 = lo;
    q.n = hi - lo;
    q.p0 = len - q.n;
    q.keys = keys_of(a, len, a.width);
  }
  return q;
}

__device__ __forceinline__ int row_tiles(const AttentionArgs& a, const Request& q, int R) {
  return (int)(((uint32_t)q.n * (uint32_t)a.G + (R - 1)) / R);   // below 2^31 rows
}

template <bool kPrefix, int R, int KT>
__device__ __forceinline__ Tiles tiles_of(const AttentionArgs& a, const Request& q, int m) {
  Tiles t;
  if (kPrefix) {
    t.p_lo = t.p_hi = q.keys - 1;
    t.sink = t.first = 0;
    t.last = (int)(((uint32_t)q.keys + (KT - 1)) / KT);
    return t;
  }
  const uint32_t row = (uint32_t)m * R;
  const int i_lo = (int)div32(row, a.inv_G);
  const int i_end = (int)div32(row + R - 1, a.inv_G);
  const int i_hi = i_end < q.n - 1 ? i_end : q.n - 1;
  t.p_lo = q.p0 + i_lo;
  t.p_hi = q.p0 + i_hi;
  const int hi = t.p_hi + 1 < q.keys ? t.p_hi + 1 : q.keys;
  if (hi <= 0) {
    t.sink = t.first = t.last = 0;
    return t;
  }
  t.last = (int)(((uint32_t)hi + (KT - 1)) / KT);
  const int low = a.window > 0 && t.p_lo >= a.window ? t.p_lo - a.window + 1 : 0;
  t.first = low / KT < t.last ? low / KT : t.last;
  const int sink_end = a.sinks < hi ? a.sinks : hi;
  const int st = (int)(((uint32_t)sink_end + (KT - 1)) / KT);
  t.sink = st < t.first ? st : t.first;
  return t;
}

// cost of a row tile: its key tiles, one at least (its rows are written)
__device__ __forceinline__ int cost_of(const Tiles& t) {
  const int c = t.count();
  return c > 1 ? c : 1;
}

// ---- shares ----------------------------------------------------------------------
constexpr int kThreads = 256;     // of the 16-row and the joining kernels

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int64_t lane_of(int64_t x, int lane) {   // uniform lane
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t add_dpp(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xf, false);
}

// values that all lanes hold alike, to scalar registers
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Request uniform_request(Request q) {
  q.token0 = uniform(q.token0);
  q.n = uniform(q.n);
  q.p0 = uniform(q.p0);
  q.keys = uniform(q.keys);
  return q;
}

// Inclusive sums over the wave's lanes of x >= 0: within rows of 16 lanes, then
// across them, in 32 bits where no sum can pass them.
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
  if (__ballot(x >= (1ll << 25)) == 0ull) {
    uint32_t v = (uint32_t)x;
    v = add_dpp<0x111, 0xf>(v);                    // row_shr:1, 2, 4, 8
    v = add_dpp<0x112, 0xf>(v);
    v = add_dpp<0x114, 0xf>(v);
    v = add_dpp<0x118, 0xf>(v);
    v = add_dpp<0x142, 0xa>(v);                    // row_bcast:15 into rows 1 and 3
    v = add_dpp<0x143, 0xc>(v);                    // row_bcast:31 into rows 2 and 3
    return v;
  }
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(x, d);
    if (lane >= d) x += u;
  }
  return x;
}

// exclusive prefix of v over the workgroup's kWaves waves; total in `all`
template <int kWaves>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_wave, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t x = wave_scan(v);
  __syncthreads();
  if (lane == 63) s_wave[wave] = x;
  __syncthreads();
  int64_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += s_wave[w];
    all += s_wave[w];
  }
  return before + x - v;
}

// Tiles of all row tiles of a request of mt, one request per lane.  A lane sums
// up to 4 row tiles itself; longer requests are taken one by one by the whole
// wave.
template <int R, int KT>
__device__ __forceinline__ int64_t request_cost(const AttentionArgs& a, const Request& q, int mt) {
  int64_t c = 0;
  if (mt <= 4)
    for (int m = 0; m < mt; ++m) c += cost_of(tiles_of<false, R, KT>(a, q, m));
  for (uint64_t rest = __ballot(mt > 4); rest != 0ull; rest &= rest - 1) {
    const int of = __ffsll((unsigned long long)rest) - 1, lane = threadIdx.x & 63;
    Request x;
    x.token0 = 0;
    x.n = __builtin_amdgcn_readlane(q.n, of);
    x.p0 = __builtin_amdgcn_readlane(q.p0, of);
    x.keys = __builtin_amdgcn_readlane(q.keys, of);
    const int xt = __builtin_amdgcn_readlane(mt, of);
    int64_t part = 0;
    for (int m = lane; m < xt; m += 64) part += cost_of(tiles_of<false, R, KT>(a, x, m));
    part = lane_of(wave_scan(part), 63);
    if (lane == of) c = part;
  }
  return c;
}

struct Place {
  int64_t share, pos, end;   // tiles per workgroup, this one's range
  double inv_share;
  int r, m, h, k;            // where pos is
  Request q;                 // request r
};

// Finds this workgroup's share of all tiles (those of the KV heads together)
// and where it begins.
template <bool kPrefix, int R, int KT, int kWaves, int kLeast>
__device__ __forceinline__ Place find_share(const AttentionArgs& a, int wg, int wgs,
                                            int64_t* s_wave, int64_t* s_found) {
  constexpr int kThreads = kWaves * 64;
  const int tid = threadIdx.x, lane = tid & 63;
  const int B = kPrefix ? 1 : a.B;
  const auto cost_at = [&](int r, Request& q) -> int64_t {   // per KV head
    q = {};
    if (r >= B) q.n = 0;
    else q = load_request<kPrefix>(a, r);
    const int mt = row_tiles(a, q, R);
    if (kPrefix) return mt > 0 ? (int64_t)mt * cost_of(tiles_of<true, R, KT>(a, q, 0)) : 0;
    return request_cost<R, KT>(a, q, mt);
  };
  Place p;
  p.r = p.m = p.h = p.k = 0;
  Request q;
  int64_t c = 0, upto = 0, total = 0;              // of this lane's request; of all
  const bool one_wave = B <= 64;                   // every wave takes all requests
  if (kPrefix) {
    total = cost_at(0, q);
  } else if (one_wave) {
    c = cost_at(lane, q);
    upto = wave_scan(c);
    total = lane_of(upto, 63);
  } else {
    for (int r0 = 0; r0 < B; r0 += kThreads) {
      int64_t all;
      block_scan<kWaves>(cost_at(r0 + tid, q), s_wave, all);
      total += all;
    }
  }
  total *= a.Hk;
  total = uniform64(total);
  p.share = uniform64(div64(total + wgs - 1, 1.0 / (double)wgs));
  p.share = p.share > kLeast ? p.share : kLeast;
  p.inv_share = __builtin_bit_cast(
      double, uniform64(__builtin_bit_cast(int64_t, 1.0 / (double)p.share)));
  p.pos = p.share * wg;
  p.end = p.pos + p.share < total ? p.pos + p.share : total;
  p.q = uniform_request(q);
  if (p.pos >= p.end) return p;
  if (kPrefix) {
    const int64_t each = cost_of(tiles_of<true, R, KT>(a, q, 0));
    p.m = uniform((int)div64(p.pos, 1.0 / (double)(each * a.Hk)));
    const int64_t x = p.pos - (int64_t)p.m * each * a.Hk;
    p.h = uniform((int)div64(x, 1.0 / (double)each));
    p.k = uniform((int)(x - p.h * each));
    return p;
  }
  int64_t x;                                       // tiles into request r
  if (one_wave) {
    const int of = __ffsll((unsigned long long)__ballot(p.pos < upto * a.Hk)) - 1;
    p.r = of;
    x = p.pos - lane_of(upto - c, of) * a.Hk;
    p.q.token0 = __builtin_amdgcn_readlane(q.token0, of);
    p.q.n = __builtin_amdgcn_readlane(q.n, of);
    p.q.p0 = __builtin_amdgcn_readlane(q.p0, of);
    p.q.keys = __builtin_amdgcn_readlane(q.keys, of);
  } else {
    int64_t base = 0;
    for (int r0 = 0; r0 < B; r0 += kThreads) {
      int64_t all;
      c = cost_at(r0 + tid, q);
      const int64_t into = p.pos - base - block_scan<kWaves>(c, s_wave, all) * a.Hk;
      if (into >= 0 && into < c * a.Hk) {          // one thread of one pass
        s_found[0] = r0 + tid;
        s_found[1] = into;
      }
      base += all * a.Hk;
      if (p.pos < base) break;                     // uniform
    }
    __syncthreads();
    p.r = uniform((int)s_found[0]);
    x = s_found[1];
    p.q = load_request<false>(a, p.r);
  }
  p.r = uniform(p.r);
  p.q = uniform_request(p.q);
  const int mt = row_tiles(a, p.q, R);
  for (int m0 = 0; m0 < mt; m0 += 64) {            // every wave alike
    const int m = m0 + lane;
    const int64_t mine = m < mt ? cost_of(tiles_of<false, R, KT>(a, p.q, m)) : 0;
    const int64_t all = wave_scan(mine);
    const uint64_t beyond = __ballot(x < all * a.Hk);
    if (beyond != 0ull) {
      const int of = __ffsll((unsigned long long)beyond) - 1;
      const int64_t each = lane_of(mine, of);
      x -= (lane_of(all, of) - each) * a.Hk;
      p.m = m0 + of;
      p.h = uniform((int)div64(x, 1.0 / (double)each));
      p.k = uniform((int)(x - p.h * each));
      break;
    }
    x -= lane_of(all, 63) * a.Hk;
  }
  return p;
}

// ---- paging ----------------------------------------------------------------------
// The cache slot of key j, whose block the table's entry names, -1 where none is
// mapped.  The entry is read ahead, while other work is done.
__device__ __forceinline__ int slot_of(int entry, int j, int page, double inv_page,
                                       int num_blocks) {
  const int i = (int)div32((uint32_t)j, inv_page);
  return entry >= 0 && entry < num_blocks ? entry * page + (j - i * page) : -1;
}

// ---- conversions -----------------------------------------------------------------
__device__ __forceinline__ bf16x8 bf16_of_codes(uint32_t w0, uint32_t w1) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f16x8 f16_of_codes(uint32_t w0, uint32_t w1) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Bytes of four dwords transposed: o[b] holds byte b of w0 .. w3.
__device__ __forceinline__ void transpose4(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3,
                                           uint32_t o[4]) {
  const uint32_t lo01 = __builtin_amdgcn_perm(w1, w0, 0x05010400u);  // a0 b0 a1 b1
  const uint32_t hi01 = __builtin_amdgcn_perm(w1, w0, 0x07030602u);  // a2 b2 a3 b3
  const uint32_t lo23 = __builtin_amdgcn_perm(w3, w2, 0x05010400u);
  const uint32_t hi23 = __builtin_amdgcn_perm(w3, w2, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
}

// nonzero iff one of the four codes is a NaN (S.1111.111)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// two fp32 to bf16, round to nearest even, in one instruction
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// what exponents are taken against: rows that have seen no key (m = -inf) take
// 0, so that exp2(-inf - 0) = 0 and nothing turns NaN
__device__ __forceinline__ float base_of(float m) { return m == FP8_NEG_INF ? 0.0f : m; }

// The base m that a row's P = exp2(score - m), l and O are kept against.  It moves
// where the row's maximum passes it by kReach, to kBelow under the maximum: the
// largest P lies in 2^kBelow .. 2^kReach, fp16's upper end, and what is lost where
// fp16 is subnormal, 2^-25, is 2^-35 of the largest weight.  Many small weights count
// together: with m at the maximum (2^-25), 131071 keys 17.4 nats below an attention
// sink, 0.0036 of the result, were all rounded to zero.  O is rescaled a few times
// per item, as the maximum may grow by 2^5 before; 12 in place of 10 takes 1.3 %
// longer for 8001 windowed tokens (64 + 8 heads of 64), 7 no less time than 10.
constexpr float kBelow = 10.0f, kReach = 15.0f;
// score - m is one fused operation, so that a score's product with its factor is
// not rounded.  The maximum is: from 2^20 on it may differ from the exact product by
// more than 2^-4, later by hundreds, and exp2 of that is no weight any more.  Where a
// wave's base gets that large (of either sign), its tiles' scores are rounded to fp32
// first, as the maximum is, and the base is the maximum itself.  A row whose base is
// not has no weight from a score that is.  `reach` then sends every tile of the item
// through the branch that moves the base, so that the others pay nothing for it.
__device__ __forceinline__ bool huge(float x) {    // 2^20 < |x| < inf
  constexpr uint32_t k = 0x49800001u;
  return (__float_as_uint(x) & 0x7fffffffu) - k < 0x7f800000u - k;
}
__device__ __forceinline__ float moved_base(float m, float top) {
  return __builtin_fmaxf(m, huge(top) ? top : top - kBelow);
}

// The keys that a row sees: lo .. hi and 0 .. sinks - 1 (up to hi).
struct Sight {
  int lo, hi, sinks;
  __device__ __forceinline__ bool sees(int j) const {
    return (j <= hi) & ((j >= lo) | (j < sinks));
  }
};
template <bool kPrefix>
__device__ __forceinline__ Sight sight_of(const AttentionArgs& a, const Request& q, int i) {
  Sight s;
  s.hi = kPrefix ? q.keys - 1 : q.p0 + i;
  s.hi = s.hi < q.keys ? s.hi : q.keys - 1;
  s.lo = !kPrefix && a.window > 0 && q.p0 + i >= a.window ? q.p0 + i - a.window + 1 : 0;
  s.sinks = a.sinks;
  return s;
}

// Arguments read again from the kernel's argument segment: what only an item's
// end needs does not stay in scalar registers through its loop.
struct KernelArgs {
  AttentionArgs a;
  Parts parts;
};
template <typename T>
__device__ __forceinline__ T* in_global(T* p) {    // tells that p is not in LDS or scratch
  const auto* any = (const __attribute__((address_space(0))) void*)p;
  __builtin_assume(!__builtin_amdgcn_is_shared(any) && !__builtin_amdgcn_is_private(any));
  return p;
}
__device__ __forceinline__ KernelArgs fresh_args() {
  typedef const __attribute__((address_space(4))) uint32_t* Words;   // scalar loads
  Words w = (Words)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(w));
  struct Raw {
    uint32_t w[sizeof(KernelArgs) / 4];
  } raw;
#pragma unroll
  for (unsigned i = 0; i < sizeof(KernelArgs) / 4; ++i) raw.w[i] = w[i];
  KernelArgs k = __builtin_bit_cast(KernelArgs, raw);
  k.a.q = in_global(k.a.q);
  k.a.kc = in_global(k.a.kc);
  k.a.vc = in_global(k.a.vc);
  k.a.table = in_global(k.a.table);
  k.a.lens = in_global(k.a.lens);
  k.a.offsets = in_global(k.a.offsets);
  k.a.prefix_table = in_global(k.a.prefix_table);
  k.a.prefix_len = in_global(k.a.prefix_len);
  k.a.v_scale = in_global(k.a.v_scale);
  k.a.out = in_global(k.a.out);
  k.a.lse = in_global(k.a.lse);
  k.parts.ml = in_global(k.parts.ml);
  k.parts.o = in_global(k.parts.o);
  k.parts.split = in_global(k.parts.split);
  k.parts.where = in_global(k.parts.where);
  k.parts.reset = in_global(k.parts.reset);
  k.parts.whole_ml = in_global(k.parts.whole_ml);
  k.parts.whole_o = in_global(k.parts.whole_o);
  return k;
}

// score factor and query sign: queries are negated (exactly) where the factor
// is negative, so that the largest score is the largest product; a factor of 0
// becomes one whose products vanish beside any maximum
struct Factor {
  float c;
  uint32_t flip;                 // xor mask of two bf16 queries
};
__device__ __forceinline__ Factor factor_of(const AttentionArgs& a) {
  const float c = a.scale * a.k_scale[0] * kLog2e;
  Factor f;
  f.c = c == 0.0f ? 0x1p-126f : __builtin_fabsf(c);
  f.flip = c < 0.0f ? 0x80008000u : 0u;
  return f;
}

__device__ __forceinline__ bf16x8 load_query(const uint16_t* p, uint32_t flip) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  return __builtin_bit_cast(bf16x8, make_uint4(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip));
}

// NaN codes of a row of D values as bits: bit e of word w is value 32 w + e
template <int kWords>
struct NanBits {
  uint32_t w[kWords];
};

// adds the NaN codes among 32 kWords bytes at p
template <int kWords>
__device__ __forceinline__ void add_nans(NanBits<kWords>& bits, const uint8_t* p) {
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    uint32_t got = 0u;
#pragma unroll 1
    for (int i = 7; i >= 0; --i) {
      const uint32_t x = nan_codes(*reinterpret_cast<const uint32_t*>(p + 32 * w + 4 * i)) >> 7;
      // bits 0, 8, 16, 24 together
      got = got << 4 | ((x | x >> 7 | x >> 14 | x >> 21) & 0xfu);
    }
    bits.w[w] |= got;
  }
}

// bytes of w that are NaN codes, cleared
__device__ __forceinline__ uint32_t without_nans(uint32_t w) {
  return w & ~((nan_codes(w) >> 7) * 0xffu);
}

// Where a workgroup's results of an item go.
struct Target {
  bool whole, begins, ends;
  int slot;                      // partial slot
  int parts;                     // workgroups that hold a part (0: whole)
};
__device__ __forceinline__ Target target_of(const Place& at, int k1, int cost, int wg) {
  Target t;
  t.begins = at.k == 0;
  t.ends = k1 == cost;
  t.whole = t.begins && t.ends;
  t.slot = 2 * wg + (t.begins ? 1 : 0);
  t.parts = t.whole ? 0 : (int)div64(at.pos + cost - 1, at.inv_share) - wg + 1;
  return t;
}

template <bool kPrefix, bool kJoin>
__device__ __forceinline__ void note_item(const Parts& parts, const Target& t, const Request& q,
                                          int row0, int rows, int head, int wg) {
  if (!kJoin && t.begins && !t.ends && threadIdx.x == 0) {
    Split s;
    s.token0 = q.token0;
    s.row0 = row0;
    s.rows = rows;
    s.head = head;
    s.parts = t.parts;
    parts.split[wg] = s;
  }
}

// m and l of a row that goes to the workspace, and where it went
template <bool kPrefix, bool kJoin>
__device__ __forceinline__ void note_row(const Parts& parts, const Target& t, int64_t flat,
                                         int part_row, float m, float l) {
  float* pm = t.whole ? parts.whole_ml + flat * 2 : parts.ml + (int64_t)part_row * 2;
  pm[0] = m;
  pm[1] = l;
  if (kJoin && t.begins) {
    parts.where[flat] = make_int2(part_row, t.parts);
    if (kPrefix) parts.reset[flat] = make_int2(0, -1);
  }
}

// ---- few rows: 16-row tiles -----------------------------------------------------
// One workgroup of 4 waves; a key tile is 128 keys, 32 per wave.  Every wave
// holds the same 16 query rows and its own m, l, O over its own keys; the four
// are joined in LDS once per item.  K and V go from memory to registers, no
// LDS: a wave reads 16 keys' rows of D bytes as whole lines (lane (n, g): D / 4
// bytes of key n), and for V lane (n, g) reads bytes n D/16 .. of the 8 keys
// that its P values stand for, transposes them in registers and converts.  The
// next unit's 8 KB (D = 128) are in flight while one is computed.
//
// Bound by the reads of the cache.  Two workgroups per CU (D = 256, whose waves
// need more registers: one) keep 64 KB in flight on a CU; loads that do not stay
// in the L2, each code being read once, gain 3 %.  64 requests of 1000 .. 8192
// keys (603 MB, D = 128) take 128 us, 4.7 TB/s; a plain sum over as many bytes
// takes 105.  One request of 131071 keys (268 MB) takes 62 us: 53 for the keys
// and 7 for the launch that joins its 512 parts.
constexpr int kRowsD = 16;
constexpr int kKeysD = 128;

template <int D>
struct Unit {
  uint32_t k[2][D / 16];   // lane (n, g): 16 bytes at 64 i + 16 g of keys n and 16 + n
  uint32_t v[8][D / 64];   // lane (n, g): D/16 bytes at n D/16 of keys 4g+i, 16+4g+i
};

// kc, vc: this lane's bytes of slot 0.  kQuads: blocks of a multiple of 4
// tokens, so that keys 4 i .. 4 i + 3 lie behind one another.
template <int D, bool kQuads>
__device__ __forceinline__ void load_unit(Unit<D>& u, const uint8_t* kc, const uint8_t* vc,
                                          uint32_t stride, int slot) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int s = __shfl(slot, 16 * t + n);
    const uint8_t* p = kc + (uint64_t)(uint32_t)(s < 0 ? 0 : s) * stride;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 64 * i));
      u.k[t][4 * i] = x.x;
      u.k[t][4 * i + 1] = x.y;
      u.k[t][4 * i + 2] = x.z;
      u.k[t][4 * i + 3] = x.w;
    }
  }
  const uint8_t* p = nullptr;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (kQuads && e % 4 != 0) {
      p += stride;
    } else {
      const int s = __shfl(slot, (e < 4 ? 0 : 12) + 4 * g + e);
      p = vc + (uint64_t)(uint32_t)(s < 0 ? 0 : s) * stride;
    }
    if constexpr (D == 64) {
      u.v[e][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (D == 128) {
      const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
      u.v[e][0] = x.x;
      u.v[e][1] = x.y;
    } else {
      const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
      u.v[e][0] = x.x;
      u.v[e][1] = x.y;
      u.v[e][2] = x.z;
      u.v[e][3] = x.w;
    }
  }
}

// V operands of one dword column of the unit: v16[b][e] = byte b of key e
__device__ __forceinline__ void v_operands(const uint32_t w[8], f16x8 out[4]) {
  uint32_t lo[4], hi[4];
  transpose4(w[0], w[1], w[2], w[3], lo);
  transpose4(w[4], w[5], w[6], w[7], hi);
#pragma unroll
  for (int b = 0; b < 4; ++b) out[b] = f16_of_codes(lo[b], hi[b]);
}

template <int D, bool kPrefix, bool kJoin, bool kQuads>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attention_rows_kernel(
    KernelArgs args) {
  constexpr int R = kRowsD, KT = kKeysD, OT = D / 16;
  constexpr int kPitch = D + 4;                    // floats: rows start in other banks
  constexpr int kNanWords = D >= 128 ? D / 128 : 1;   // of a lane's D / 4 values
  __shared__ float s_o[4][R][kPitch];
  __shared__ float s_ml[4][R][2];
  __shared__ int64_t s_wave[4], s_found[2];
  const AttentionArgs& a = args.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int wg = blockIdx.x;
  Place at = find_share<kPrefix, R, KT, 4, 2>(a, wg, gridDim.x, s_wave, s_found);
  if (!kJoin && tid == 0) args.parts.split[wg].parts = 0;
  const uint32_t stride = (uint32_t)a.Hk * D;
  const Factor fac = factor_of(a);
  const float c = fac.c;

  while (at.pos < at.end) {
    const Request q = at.q;
    const int mt = row_tiles(a, q, R);
    if (at.m >= mt) {                              // done, or without queries
      at.q = uniform_request(load_request<kPrefix>(a, ++at.r));
      at.m = at.h = at.k = 0;
      continue;
    }
    const Tiles tl = tiles_of<kPrefix, R, KT>(a, q, at.m);
    const int cost = cost_of(tl);
    const int64_t left = at.end - at.pos;
    const int k1 = uniform((int64_t)(cost - at.k) < left ? cost : at.k + (int)left);
    const int row0 = at.m * R;
    const int rest = q.n * a.G - row0;
    const int rows = uniform(rest < R ? rest : R);

    // this lane's row: queries of row n, k slices of group g
    const int i_n = n < rows ? (int)div32((uint32_t)(row0 + n), a.inv_G) : 0;
    const Sight sight = sight_of<kPrefix>(a, q, i_n);
    bf16x8 qf[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qf[i] = bf16x8{};
    if (n < rows) {
      const uint16_t* p = a.q + (int64_t)(q.token0 + i_n) * a.ld_q +
                          (int64_t)(at.h * a.G + row0 + n - i_n * a.G) * D + g * 16;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        qf[i] = load_query(p + 64 * (i / 2) + 8 * (i % 2), fac.flip);
    }
    float m = FP8_NEG_INF, l = 0.0f;
    float base = 0.0f, reach = kReach;             // base: of m, what is subtracted
    f32x4 o[OT];
#pragma unroll
    for (int j = 0; j < OT; ++j) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    NanBits<kNanWords> nans = {};

    const int count = tl.count();
    const int kend = k1 < count ? k1 : count;      // an item of no keys has no tile
    if (at.k < kend) {
      const int32_t* table = kPrefix ? a.prefix_table : a.table + (int64_t)at.r * a.ld_table;
      const uint8_t* kc = a.kc + (int64_t)at.h * D + g * 16;
      const uint8_t* vc = a.vc + (int64_t)at.h * D + n * (D / 16);
      auto key_at = [&](int k) { return tl.key_tile(k) * KT + wave * 32 + (lane & 31); };
      // read without a branch (the last key's where there is none), so that
      // nothing waits for it before its use
      auto entry_at = [&](int k) {
        const int j = key_at(k);
        return table[div32((uint32_t)(j < q.keys ? j : q.keys - 1), a.inv_page)];
      };
      auto slot_at = [&](int k, int entry) {
        const int j = key_at(k);
        return slot_of(k < kend && j < q.keys ? entry : -1, j, a.page, a.inv_page, a.num_blocks);
      };
      // while a unit is computed the next one's codes are in flight
      Unit<D> unit[2];
      int slot = slot_at(at.k, entry_at(at.k)), entry = entry_at(at.k + 1);
      load_unit<D, kQuads>(unit[0], kc, vc, stride, slot);
      auto step = [&](int k, Unit<D>& now, Unit<D>& next) {
        const int kb = tl.key_tile(k) * KT + wave * 32;
        const int mine = slot;
        slot = slot_at(k + 1, entry);
        entry = entry_at(k + 2);
        load_unit<D, kQuads>(next, kc, vc, stride, slot);
        const uint32_t mapped = (uint32_t)__ballot(mine >= 0);
        if (mapped == 0u) return;                  // nothing of these 32 keys is there
        // S^T: keys 16 t + 4 g + i of row n
        f32x4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                bf16_of_codes(now.k[t][2 * i], now.k[t][2 * i + 1]), qf[i], s[t], 0, 0, 0);
        }
        const int last = kb + 31;
        const bool all = mapped == 0xffffffffu && last <= tl.p_lo &&
                         (a.window == 0 || tl.p_hi - kb < a.window || last < a.sinks);
        if (!all) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int b = 16 * t + 4 * g + i;
              const bool v = ((mapped >> b) & 1u) & (uint32_t)sight.sees(kb + b);
              s[t][i] = v ? s[t][i] : FP8_NEG_INF;
            }
          // values that are not there are zeros
          uint32_t nan = 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool there = (mapped >> ((e < 4 ? 0 : 12) + 4 * g + e)) & 1u;
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              now.v[e][w] = there ? now.v[e][w] : 0u;
              nan |= nan_codes(now.v[e][w]);
            }
          }
          // a NaN that some rows see and others do not: a zero here, and
          // noted for the rows that see it
          if (__ballot(nan != 0u) != 0ull) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
              for (int w = 0; w < D / 64; ++w) now.v[e][w] = without_nans(now.v[e][w]);
#pragma unroll 1
            for (int b = 0; b < 32; ++b) {
              const int sb = __shfl(mine, b);
              if (sb >= 0 && sight.sees(kb + b)) {
                const uint8_t* p = a.vc + (int64_t)at.h * D + (uint64_t)(uint32_t)sb * stride +
                                   g * (D / 4);
                if constexpr (D >= 128) {
                  add_nans(nans, p);
                } else {                           // 16 values of a lane
#pragma unroll 1
                  for (int i = 0; i < 16; ++i)
                    nans.w[0] |= (uint32_t)((p[i] & 0x7fu) == 0x7fu) << i;
                }
              }
            }
          }
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, s[t][i]);
        top = max_xor32(max_xor16(top)) * c;
        if (__ballot(top - m > reach) != 0ull) {  // some row's maximum grew out of reach
          const float m_new = moved_base(m, top);
          const float alpha = __builtin_amdgcn_exp2f(m - base_of(m_new));
          l *= alpha;
#pragma unroll
          for (int j = 0; j < OT; ++j) o[j] *= alpha;
          m = m_new;
          base = base_of(m);
          if (__ballot(huge(m)) != 0ull) {         // see huge
            reach = FP8_NEG_INF;
            const float inv = 1.0f / c;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[t][i] = (s[t][i] * c - base) * inv;
            base = 0.0f;
          }
        }
        float sum = 0.0f;
        f16x8 p;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c, -base));
            sum += e;
            p[4 * t + i] = (_Float16)e;
          }
        l += sum;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t col[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) col[i] = now.v[i][w];
          f16x8 vo[4];
          v_operands(col, vo);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            o[4 * w + b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vo[b], p, o[4 * w + b], 0, 0, 0);
        }
      };
#pragma unroll 1
      for (int k = at.k;;) {
        step(k, unit[0], unit[1]);
        if (++k >= kend) break;
        step(k, unit[1], unit[0]);
        if (++k >= kend) break;
      }
    }
    l = sum_xor32(sum_xor16(l));

    // join the four waves: lane (n, g) holds d = (4 g + i) OT + j of row n
    __syncthreads();                               // the last item's readers are done
    if (n < rows) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < OT; j += 4) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int bit = i * OT + j + e;        // of this lane's D / 4 values
            x[e] = (nans.w[bit / 32] >> (bit % 32)) & 1u ? __builtin_nanf("") : o[j + e][i];
          }
          *reinterpret_cast<float4*>(&s_o[wave][n][(4 * g + i) * OT + j]) =
              make_float4(x[0], x[1], x[2], x[3]);
        }
      if (g == 0) {
        s_ml[wave][n][0] = m;
        s_ml[wave][n][1] = l;
      }
    }
    __syncthreads();
    const KernelArgs fr = fresh_args();
    const Parts parts = fr.parts;
    const Target to = target_of(at, k1, cost, wg);
    // a thread takes 4 values of a row at a time
    constexpr int kVec = D / 4;
    for (int x = tid; x < rows * kVec; x += kThreads) {
      const int row = x / kVec, d = (x - row * kVec) * 4;
      float mm = s_ml[0][row][0];
#pragma unroll
      for (int w = 1; w < 4; ++w) mm = __builtin_fmaxf(mm, s_ml[w][row][0]);
      const float base = base_of(mm);
      float ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_ml[w][row][0] - base);
        ll = __builtin_fmaf(s_ml[w][row][1], f, ll);
        const float4 y = *reinterpret_cast<const float4*>(&s_o[w][row][d]);
        acc[0] = __builtin_fmaf(y.x, f, acc[0]);
        acc[1] = __builtin_fmaf(y.y, f, acc[1]);
        acc[2] = __builtin_fmaf(y.z, f, acc[2]);
        acc[3] = __builtin_fmaf(y.w, f, acc[3]);
      }
      const int rr = row0 + row, i = (int)div32((uint32_t)rr, a.inv_G);
      const int64_t token = q.token0 + i;
      const int head = at.h * a.G + rr - i * a.G;
      const int64_t flat = token * a.Hq + head;
      if (to.whole && !kJoin) {
        const float inv = ll == 0.0f ? 0.0f : fr.a.v_scale[0] / ll;
        const uint32_t w0 = pack_bf16(acc[0] * inv, acc[1] * inv);
        const uint32_t w1 = pack_bf16(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2*>(fr.a.out + token * fr.a.ld_out + (int64_t)head * D + d) =
            make_uint2(w0, w1);
        if (fr.a.lse && d == 0) fr.a.lse[flat] = (base + __builtin_log2f(ll)) * kLn2;
      } else {
        const int part_row = to.slot * R + row;
        float* po = to.whole ? parts.whole_o + flat * D : parts.o + (int64_t)part_row * D;
        *reinterpret_cast<float4*>(po + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (d == 0) note_row<kPrefix, kJoin>(parts, to, flat, part_row, mm, ll);
      }
    }
    note_item<kPrefix, kJoin>(parts, to, q, row0, rows, at.h, wg);
    at.pos += k1 - at.k;
    at.k = 0;
    if (++at.h == a.Hk) {
      at.h = 0;
      ++at.m;
    }
  }
}

// ---- many rows: 256-row tiles ----------------------------------------------------
// One workgroup of 8 waves, 32 rows each; a key tile is 64 keys (128 for D = 64),
// staged in LDS once for all waves: K as bf16 [key][D], V as fp16 [d][key], both
// converted on the way in (V transposed in registers, 4 keys at a time), two
// buffers each.  256 rows a tile, so that the conversion of a code (which costs as
// much as its product with 32 rows) and its read are shared by as many rows as the
// registers of a CU hold.
// 32 x 32 x 16 products: lane (n, g) with n = lane % 32 holds row n of S^T and O^T.
//
// Two phases alternate: products (V j with P j, then K j + 1 with Q) and softmax
// (S j to P j).  The waves form two groups half a period apart, a barrier between
// the phases: while one group keeps a SIMD's matrix unit busy, the other, on the
// same SIMD, has its vector unit.  A wave issues a vector instruction every 7
// cycles beside another's products, so what else there is to do stands between
// the products, 32 cycles each: parts of K j + 2 and V j + 1 go from registers to
// LDS, and the codes behind them are read.  With j counting tiles, interval i
// between two barriers holds softmax j of the first group at i = 2 j + 1 and its
// products j at 2 j + 2, those of the second group one interval later.  K j + 1
// and V j are then read in 2 j + 2 and 2 j + 3; they were written in the two
// intervals before, when their buffers' last readers were done.
//
// Bound by the longer phase, twice per tile, as the groups are half a period apart.
// Measured at D = 128, per tile of 64 keys and wave: products 1880 cycles (1024 of
// them the matrix unit's, the rest operands from LDS and the staging in between),
// softmax 1390 and 450 of waiting for the other group's products; two waves on a
// SIMD then use 55 % of its matrix unit.  At D = 64, per tile of 128 keys, softmax
// is the longer one, 2550 to 1950.  An item's start and end, 25000 cycles where
// nothing overlaps, weigh as 6 to 7 tiles.  8192 tokens of 3 requests behind up to
// 4096 cached ones (32 + 8 heads of 128, 519 GFLOP in visible pairs) take 616 to
// 670 us, 0.8 PFLOP/s, where a large bf16 matrix product reaches 1.42.  8001 tokens
// with a window of 1000 (64 + 8 heads of 64, 132 GFLOP) take 306: tiles that the
// mask cuts are computed whole, and a key's softmax stands beside half the products.
//
// LDS rows are cut into 16-byte pieces whose index is XORed with the row's, so
// that the 32 rows that one read names lie in different banks.  O^T's rows
// are not d in order: row 32 b + 8 i + 4 g + e is d = g D/2 + 16 b + 4 i + e, which
// leaves each lane with D / 2 values in a row to store.
constexpr int tile_keys(int D) { return D == 64 ? 128 : 64; }

constexpr int kTileWaves = 8;

template <int D, bool kPrefix, bool kJoin>
__global__ __launch_bounds__(kTileWaves * 64, 2) void attention_tile_kernel(KernelArgs args) {
  static_assert(D <= 128, "a wave's registers");
  constexpr int kWaves = kTileWaves;
  constexpr int R = kWaves * 32, KT = tile_keys(D);
  constexpr int KS = D / 16;                       // k steps of K Q^T
  constexpr int OB = D / 32;                       // 32-row blocks of O^T
  constexpr int NB = KT / 32;                      // 32-key blocks of S^T
  constexpr int kThreads = kWaves * 64;
  constexpr int TK = kThreads / KT;                // threads of a key's row of K
  constexpr int TV = kThreads / (KT / 4);          // threads of four keys' rows of V
  constexpr int KW = D / TK / 4;                   // dwords that one takes of the row of K
  static_assert(D / TV == 4, "one of each of the rows of V");
  constexpr int kBuf = KT * D * 2;                 // bytes of a K or V buffer
  constexpr int kPieces = D / 8 < 16 ? D / 8 - 1 : 15;   // K's XOR range
  __shared__ __attribute__((aligned(16))) uint8_t s_kv[4 * kBuf];   // K0 K1 V0 V1
  __shared__ __attribute__((aligned(16))) int s_slot[8][KT];   // of tile k in s_slot[k % 8]
  __shared__ int s_nan[2];                         // the last tile staged there with a NaN value
  __shared__ int64_t s_wave[kWaves], s_found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int n = lane & 31, g = lane >> 5;
  const bool second = wave >= kWaves / 2;          // group
  // neighbouring shares, which read the same keys, on one XCD (workgroups go
  // round robin over the 8)
  const int wgs = gridDim.x;
  const int wg = wgs % 8 == 0 ? (int)(blockIdx.x % 8) * (wgs / 8) + (int)(blockIdx.x / 8)
                              : (int)blockIdx.x;
  Place at = find_share<kPrefix, R, KT, kWaves, 1>(args.a, wg, wgs, s_wave, s_found);
  if (!kJoin && tid == 0) args.parts.split[wg].parts = 0;
  const uint32_t stride = (uint32_t)args.a.Hk * D;
  const Factor fac = factor_of(args.a);
  const float c = fac.c;

  // LDS places of this thread in buffers 0.  Reads: piece of k step 0 of row n of
  // K and of V; step i XORs 2 i.
  const uint32_t from_k = n * (2 * D) + (g ^ (n & kPieces)) * 16;
  const uint32_t from_v = 2 * kBuf + n * (2 * KT) + (g ^ ((n ^ (n >> 3)) & 7)) * 16;
  // Writes: a thread puts 4 KW codes of key tid / TK, and of each of its 4 V
  // columns half a piece, keys first_v .. + 3.  Column e is V row r0 + e (see the
  // order of O^T's rows above), whose pieces' index XORs e.
  const int key_k = tid / TK, x_v = tid % TV, y_v = tid / TV;
  const uint32_t to_k =
      key_k * (2 * D) + (((tid % TK) * (KW / 2)) ^ (key_k & kPieces)) * 16;
  const int first_v = (y_v >> 2) * 16 + ((y_v >> 1) & 1) * 4 + (y_v & 1) * 8;
  const int rem_v = x_v * 4 % (D / 2);
  const int r0_v = (rem_v / 16) * 32 + ((rem_v / 4) % 4) * 8 + (x_v / (TV / 2)) * 4;
  const uint32_t to_v = 2 * kBuf + r0_v * (2 * KT) +
                        ((y_v >> 1) ^ ((r0_v ^ (r0_v >> 3)) & 7)) * 16 + (y_v & 1) * 8;

  while (at.pos < at.end) {
    const AttentionArgs a = fresh_args().a;        // see there
    const Request q = at.q;
    const int mt = row_tiles(a, q, R);
    if (at.m >= mt) {                              // done, or without queries
      at.q = uniform_request(load_request<kPrefix>(a, ++at.r));
      at.m = at.h = at.k = 0;
      continue;
    }
    const Tiles tl = tiles_of<kPrefix, R, KT>(a, q, at.m);
    const int cost = cost_of(tl);
    const int64_t left = at.end - at.pos;
    const int k1 = uniform((int64_t)(cost - at.k) < left ? cost : at.k + (int)left);
    const int row0 = at.m * R;
    const int rest = q.n * a.G - row0;
    const int rows = uniform(rest < R ? rest : R);

    const int row = wave * 32 + n;                 // this lane's row of the tile
    const bool mine = row < rows;
    const int i_n = mine ? (int)div32((uint32_t)(row0 + row), a.inv_G) : 0;
    const Sight sight = sight_of<kPrefix>(a, q, i_n);
    bf16x8 qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] = bf16x8{};
    if (mine) {
      const uint16_t* p = a.q + (int64_t)(q.token0 + i_n) * a.ld_q +
                          (int64_t)(at.h * a.G + row0 + row - i_n * a.G) * D + g * 8;
#pragma unroll
      for (int i = 0; i < KS; ++i) qf[i] = load_query(p + 16 * i, fac.flip);
    }
    // from the kernel's own parameters, which are known to point to memory
    const int32_t* table =
        kPrefix ? args.a.prefix_table : args.a.table + (int64_t)at.r * a.ld_table;
    const uint8_t* vc = args.a.vc + (int64_t)at.h * D;
    const uint8_t* codes_k = args.a.kc + (int64_t)at.h * D + (tid % TK) * (4 * KW);   // this thread's
    const uint8_t* codes_v = vc + x_v * 4;
    const int count = tl.count();
    const int kend = k1 < count ? k1 : count;
    float m, l;
    float base, reach;                             // base: of m, what is subtracted
    f32x16 o[OB];
    NanBits<D / 64> nans;                          // of this lane's D / 2 values

    // A NaN code among the values makes O NaN in every row of the tile, also in
    // rows that do not see it.  That is found at the end, and the item is then
    // done again with the values' codes looked at: NaNs enter as zeros, and the
    // rows that see them note which.
    for (bool careful = false;; careful = true) {
      m = FP8_NEG_INF;
      l = 0.0f;
      base = 0.0f;
      reach = kReach;
      nans = {};
#pragma unroll
      for (int b = 0; b < OB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;
      uint32_t raw_k[KW], raw_v[4];
      // The table's entry and the slot of key tid % KT of tile k.  The entry is
      // read without a branch (of the last key where there is none), so that
      // nothing waits for it before its use.
      auto key_at = [&](int k) { return tl.key_tile(k) * KT + tid % KT; };
      auto entry_at = [&](int k) {
        const int j = key_at(k);
        return table[div32((uint32_t)(j < q.keys ? j : q.keys - 1), a.inv_page)];
      };
      auto slot_at = [&](int k, int entry) {
        const int j = key_at(k);
        return slot_of((k < kend) & (j < q.keys) ? entry : -1, j, a.page, a.inv_page, a.num_blocks);
      };
      // Codes to registers: part i of a thread's piece of a key, and what it
      // takes of one of four keys' values.
      constexpr int kLoads = KW / 4 + 4;
      auto fetch_k = [&](int i, int slot) {
        const uint8_t* p = codes_k + (uint64_t)(uint32_t)(slot < 0 ? 0 : slot) * stride;
        const uint4 x = *reinterpret_cast<const uint4*>(p + 16 * i);
        raw_k[4 * i] = x.x;
        raw_k[4 * i + 1] = x.y;
        raw_k[4 * i + 2] = x.z;
        raw_k[4 * i + 3] = x.w;
      };
      auto fetch_v = [&](int e, const int4& slots) {
        const int slot = e == 0 ? slots.x : e == 1 ? slots.y : e == 2 ? slots.z : slots.w;
        const uint8_t* p = codes_v + (uint64_t)(uint32_t)(slot < 0 ? 0 : slot) * stride;
        raw_v[e] = *reinterpret_cast<const uint32_t*>(p);
      };
      auto slot_k = [&](int k) { return s_slot[k & 7][key_k]; };
      auto slots_v = [&](int k) {
        return *reinterpret_cast<const int4*>(&s_slot[k & 7][first_v]);
      };
      // A key of tile k per lane (and 64 behind it): its slot
      auto lane_slots = [&](int k, int x[NB / 2]) {
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) x[i] = s_slot[k & 7][64 * i + lane];
      };
      // Whether a key of tile k is not there; whether one before the last key is
      // not, that is, in an unmapped page.
      auto any_gap = [&](const int x[NB / 2]) {
        bool gap = x[0] < 0;
#pragma unroll
        for (int i = 1; i < NB / 2; ++i) gap |= x[i] < 0;
        return __ballot(gap) != 0ull;
      };
      auto any_hole = [&](int k, const int x[NB / 2]) {
        const int j = tl.key_tile(k) * KT + lane;
        bool hole = (x[0] < 0) & (j < q.keys);
#pragma unroll
        for (int i = 1; i < NB / 2; ++i) hole |= (x[i] < 0) & (j + 64 * i < q.keys);
        return __ballot(hole) != 0ull;
      };
      // Rare: values of keys that are not there become zeros, whatever the
      // address held, and a careful pass takes the NaNs out.
      auto mend_v = [&](int k, int buf, bool gap) {
        if (gap) {
          const int4 sv = slots_v(k);
          const int s4[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) raw_v[e] = s4[e] < 0 ? 0u : raw_v[e];
        }
        if (careful) {
          uint32_t nan = 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) nan |= nan_codes(raw_v[i]);
          if (nan != 0u) s_nan[buf] = k;
#pragma unroll
          for (int i = 0; i < 4; ++i) raw_v[i] = without_nans(raw_v[i]);
        }
      };
      // The codes in registers go to LDS, converted, in small steps u.
      constexpr int kPutsK = 2 * KW, kPutsV = 10;
      uint32_t col[4], half_k[4], half[4];
      auto put_k = [&](int u, uint32_t to) {        // two codes; 16 bytes every 4 steps
        const int i = u / 4, j = u % 4;
        half_k[j] = __builtin_bit_cast(
            uint32_t,
            j & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw_k[2 * i + j / 2], 1.0f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw_k[2 * i + j / 2], 1.0f, false));
        if (j == 3) {
          *reinterpret_cast<uint4*>(s_kv + (to ^ (16 * i))) =
              make_uint4(half_k[0], half_k[1], half_k[2], half_k[3]);
        }
      };
      auto put_v = [&](int u, uint32_t to) {        // a dword column of 4 keys in 10 steps
        if (u == 0) {
          half[0] = __builtin_amdgcn_perm(raw_v[1], raw_v[0], 0x05010400u);
          half[1] = __builtin_amdgcn_perm(raw_v[1], raw_v[0], 0x07030602u);
          half[2] = __builtin_amdgcn_perm(raw_v[3], raw_v[2], 0x05010400u);
          half[3] = __builtin_amdgcn_perm(raw_v[3], raw_v[2], 0x07030602u);
        } else if (u == 1) {
          col[0] = __builtin_amdgcn_perm(half[2], half[0], 0x05040100u);
          col[1] = __builtin_amdgcn_perm(half[2], half[0], 0x07060302u);
          col[2] = __builtin_amdgcn_perm(half[3], half[1], 0x05040100u);
          col[3] = __builtin_amdgcn_perm(half[3], half[1], 0x07060302u);
        } else if (u % 2 == 0) {
          half[0] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(col[u / 2 - 1], 1.0f, false));
        } else {
          const int b = u / 2 - 1;                 // column
          half[1] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(col[b], 1.0f, true));
          *reinterpret_cast<uint2*>(s_kv + (to ^ (16 * b)) + b * (2 * KT)) =
              make_uint2(half[0], half[1]);
        }
      };
      if (at.k < kend) {
        if (tid < 2) s_nan[tid] = -1;
        int entry;                                 // of tile k + 4
        {
          int first[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) first[i] = entry_at(at.k + i);
          entry = entry_at(at.k + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s_slot[(at.k + i) & 7][tid % KT] = slot_at(at.k + i, first[i]);
        }
        __syncthreads();
        // K k, K k + 1 and V k to LDS; K k + 2 and V k + 1 stay in registers
        int x[NB / 2];
        lane_slots(at.k, x);
        uint32_t k0[KW], v0[4], k1[KW];
        const auto load_k = [&](int k) {
          const int slot = slot_k(k);
#pragma unroll
          for (int i = 0; i < KW / 4; ++i) fetch_k(i, slot);
        };
        const auto load_v = [&](int k) {
          const int4 slots = slots_v(k);
#pragma unroll
          for (int e = 0; e < 4; ++e) fetch_v(e, slots);
        };
        load_k(at.k);
#pragma unroll
        for (int i = 0; i < KW; ++i) k0[i] = raw_k[i];
        load_v(at.k);
#pragma unroll
        for (int i = 0; i < 4; ++i) v0[i] = raw_v[i];
        load_k(at.k + 1);
#pragma unroll
        for (int i = 0; i < KW; ++i) k1[i] = raw_k[i];
        load_k(at.k + 2);
        load_v(at.k + 1);
        uint32_t k2[KW], v1[4];
#pragma unroll
        for (int i = 0; i < KW; ++i) k2[i] = raw_k[i], raw_k[i] = k0[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) v1[i] = raw_v[i], raw_v[i] = v0[i];
#pragma unroll
        for (int u = 0; u < kPutsK; ++u) put_k(u, to_k);
        mend_v(at.k, 0, any_gap(x));
#pragma unroll
        for (int u = 0; u < kPutsV; ++u) put_v(u, to_v);
#pragma unroll
        for (int i = 0; i < KW; ++i) raw_k[i] = k1[i];
#pragma unroll
        for (int u = 0; u < kPutsK; ++u) put_k(u, to_k + kBuf);
#pragma unroll
        for (int i = 0; i < KW; ++i) raw_k[i] = k2[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw_v[i] = v1[i];
        __syncthreads();
        if (second) __syncthreads();               // half a period behind
        // S^T: block t holds keys 32 t + 8 (v / 4) + 4 g + v % 4 of row n
        f32x16 s[NB];
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int v = 0; v < 16; ++v) s[t][v] = 0.0f;
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int t = 0; t < NB; ++t)
            s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8*>(s_kv + (from_k ^ (32 * i)) + t * (64 * D)),
                qf[i], s[t], 0, 0, 0);
        __syncthreads();
        int cur = 0;
        // tile k has unmapped keys; V k + 1 lacks some
        int x0[NB / 2], x1[NB / 2];
        lane_slots(at.k, x0);
        lane_slots(at.k + 1, x1);
        bool holes = any_hole(at.k, x0), gap = any_gap(x1);
#pragma unroll 1
        for (int k = at.k; k < kend; ++k) {
          // what is formed from these is formed in each pass: kept through the
          // loop it would take the registers that the products' operands need
          int g_ = g;
          uint32_t at_k = from_k, at_v = from_v, put_at_k = to_k, put_at_v = to_v;
          asm volatile("" : "+v"(g_), "+v"(at_k), "+v"(at_v), "+v"(put_at_k), "+v"(put_at_v));
          at_k += (cur ^ 1) * kBuf;
          at_v += cur * kBuf;
          put_at_k += cur * kBuf;
          put_at_v += (cur ^ 1) * kBuf;
          const int kb = tl.key_tile(k) * KT;
          const int last = kb + KT - 1;
          // three kinds of keys that not every row sees, each rare: behind the
          // row (or the last key), before its window, in an unmapped page
          if (last > (kPrefix ? q.keys - 1 : tl.p_lo) || last >= q.keys) {
            const int hi = sight.hi - kb - 4 * g_;
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                s[t][v] = 32 * t + 8 * (v / 4) + v % 4 <= hi ? s[t][v] : FP8_NEG_INF;
                if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // few masks at a time
              }
          }
          if (!kPrefix && a.window > 0 && tl.p_hi - kb >= a.window && last >= a.sinks) {
            const int lo = sight.lo - kb - 4 * g_, sk = sight.sinks - kb - 4 * g_;
            if (kb >= a.sinks) {
#pragma unroll
              for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                  s[t][v] = 32 * t + 8 * (v / 4) + v % 4 >= lo ? s[t][v] : FP8_NEG_INF;
                  if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            } else {
              int lo2 = lo;
              asm volatile("" : "+v"(lo2));        // its comparisons are its own
#pragma unroll
              for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                  const int j = 32 * t + 8 * (v / 4) + v % 4;
                  s[t][v] = (j >= lo2) | (j < sk) ? s[t][v] : FP8_NEG_INF;
                  if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
          }
          if (holes) {
#pragma unroll
            for (int t = 0; t < NB; ++t) {
              const uint64_t map = __ballot(s_slot[k & 7][64 * (t / 2) + lane] >= 0);
              const uint32_t there = (uint32_t)(map >> (32 * (t & 1))) >> (4 * g_);
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                s[t][v] = (there >> (8 * (v / 4) + v % 4)) & 1u ? s[t][v] : FP8_NEG_INF;
                if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
          float top = s[0][0];
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) top = __builtin_fmaxf(top, s[t][v]);
          top = max_xor32(top) * c;
          if (__ballot(top - m > reach) != 0ull) {  // some row's maximum grew out of reach
            const float m_new = moved_base(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - base_of(m_new));
            l *= alpha;
#pragma unroll
            for (int b = 0; b < OB; ++b)
#pragma unroll
              for (int i = 0; i < 16; ++i) o[b][i] *= alpha;
            m = m_new;
            base = base_of(m);
            if (__ballot(huge(m)) != 0ull) {       // see huge
              reach = FP8_NEG_INF;
              float d = c;
              asm volatile("" : "+v"(d));          // its reciprocal is not kept through the loop
              const float inv = 1.0f / d;
#pragma unroll
              for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int v = 0; v < 16; ++v) s[t][v] = (s[t][v] * c - base) * inv;
              base = 0.0f;
            }
          }
          float sum = 0.0f;
          f16x8 p[KT / 16];
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][v], c, -base));
              sum += e;
              p[2 * t + v / 8][v % 8] = (_Float16)e;
            }
          l += sum;
          // P is formed on this side of the barrier
#pragma unroll
          for (int i = 0; i < KT / 16; ++i) asm volatile("" : "+v"(p[i]));
          asm volatile("" : "+v"(l));
          __syncthreads();

          if (careful && s_nan[cur] == k) {        // NaN values: which ones does this row see?
#pragma unroll 1
            for (int b = 0; b < KT; ++b) {
              const int sb = s_slot[k & 7][b];
              if (sb >= 0 && sight.sees(kb + b))
                add_nans(nans, vc + (uint64_t)(uint32_t)sb * stride + g_ * (D / 2));
            }
          }
          __builtin_amdgcn_s_setprio(2);           // the products go first
          mend_v(k + 1, cur ^ 1, gap);
          // product e: V k with P k (k step e / OB, block e % OB), then K k + 1 with
          // Q (k step e / NB, block e % NB); operands are read kAhead products ahead
          constexpr int kPV = KT / 16 * OB, kProducts = kPV + KS * NB, kAhead = 4;
          auto operand = [&](int e) {
            if (e < kPV)
              return *reinterpret_cast<const uint4*>(
                  s_kv + (at_v ^ (32 * (e / OB)) ^ (64 * (e % OB & 1))) + (e % OB) * (64 * KT));
            e -= kPV;
            return *reinterpret_cast<const uint4*>(s_kv + (at_k ^ (32 * (e / NB))) +
                                                   (e % NB) * (64 * D));
          };
          // what stands between them, kPer steps behind each product
          constexpr int kSteps = kPutsK + kPutsV + kLoads;
          constexpr int kPer = (kSteps + kProducts - 1) / kProducts;
          const int slot = slot_k(k + 3);
          const int4 slots = slots_v(k + 2);
          lane_slots(k + 1, x0);
          lane_slots(k + 2, x1);
          // slots of tile k + 4, which every pair of waves writes alike and which
          // the products of tile k + 1 read; the entries behind them
          s_slot[(k + 4) & 7][tid % KT] = slot_at(k + 4, entry);
          entry = entry_at(k + 5);
          const f32x16 zero = {};
          uint4 f[kAhead + 1];
#pragma unroll
          for (int e = 0; e < kAhead; ++e) f[e] = operand(e);
#pragma unroll
          for (int e = 0; e < kProducts; ++e) {
            if (e + kAhead < kProducts) f[(e + kAhead) % (kAhead + 1)] = operand(e + kAhead);
            const uint4 x = f[e % (kAhead + 1)];
            if (e < kPV) {
              o[e % OB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x),
                                                                 p[e / OB], o[e % OB], 0, 0, 0);
            } else {
              const int i = (e - kPV) / NB, t = (e - kPV) % NB;
              s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), qf[i],
                                                             i == 0 ? zero : s[t], 0, 0, 0);
            }
#pragma unroll
            for (int u = e * kPer; u < (e + 1) * kPer; ++u) {
              if (u < kPutsK) put_k(u, put_at_k);
              else if (u < kPutsK + kPutsV) put_v(u - kPutsK, put_at_v);
              else if (u < kPutsK + kPutsV + KW / 4) fetch_k(u - kPutsK - kPutsV, slot);
              else if (u < kSteps) fetch_v(u - kPutsK - kPutsV - KW / 4, slots);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          holes = any_hole(k + 1, x0);
          gap = any_gap(x1);
          __builtin_amdgcn_s_setprio(0);
          __syncthreads();
          cur ^= 1;
        }
        if (!second) __syncthreads();
      }
      if (careful) break;
      bool bad = false;
#pragma unroll
      for (int b = 0; b < OB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) bad |= o[b][i] != o[b][i];
      if (!__syncthreads_or(bad)) break;
    }
    l = sum_xor32(l);

    const KernelArgs fr = fresh_args();
    const Parts parts = fr.parts;
    const Target to = target_of(at, k1, cost, wg);
    if (mine) {
      bool any = false;
#pragma unroll
      for (int w = 0; w < D / 64; ++w) any |= nans.w[w] != 0u;
      if (any) {
#pragma unroll
        for (int b = 0; b < OB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int bit = 16 * b + i;
            o[b][i] = (nans.w[bit / 32] >> (bit % 32)) & 1u ? __builtin_nanf("") : o[b][i];
          }
      }
      const int64_t flat = (int64_t)(q.token0 + i_n) * fr.a.Hq + at.h * a.G + row0 + row - i_n * a.G;
      if (g == 0) {
        if (!to.whole || kJoin) note_row<kPrefix, kJoin>(parts, to, flat, to.slot * R + row, m, l);
        else if (fr.a.lse) fr.a.lse[flat] = (base_of(m) + __builtin_log2f(l)) * kLn2;
      }
    }
    // A lane holds a row, and its stores would touch 64 lines each; the wave's
    // part of the staging buffers, which all waves are done with, turns them into
    // stores of whole rows, 16-byte pieces XORed with the row as above.
    uint8_t* turn = s_kv + wave * (4 * kBuf / kWaves);
    constexpr int kTurn = 4 * kBuf / kWaves / 32;  // bytes of a row there
    const auto out_row = [&](int r) {              // where row r of the wave goes: token, head
      const int rho = row0 + wave * 32 + r, i = (int)div32((uint32_t)rho, a.inv_G);
      return make_int2(q.token0 + i, at.h * a.G + rho - i * a.G);
    };
    if (to.whole && !kJoin) {
      const float inv = l == 0.0f ? 0.0f : fr.a.v_scale[0] / l;
      constexpr int kPieces16 = D * 2 / 16;        // of a row of bf16
      static_assert(D * 2 <= kTurn, "a row fits");
#pragma unroll
      for (int b = 0; b < OB; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          const int piece = g * (kPieces16 / 2) + 2 * b + i / 8;
          *reinterpret_cast<uint4*>(turn + n * kTurn + (piece ^ (n & 7)) * 16) =
              make_uint4(pack_bf16(o[b][i] * inv, o[b][i + 1] * inv),
                         pack_bf16(o[b][i + 2] * inv, o[b][i + 3] * inv),
                         pack_bf16(o[b][i + 4] * inv, o[b][i + 5] * inv),
                         pack_bf16(o[b][i + 6] * inv, o[b][i + 7] * inv));
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int x = 0; x < 32 * kPieces16 / 64; ++x) {
        const int r = (x * 64 + lane) / kPieces16, piece = (x * 64 + lane) % kPieces16;
        const uint4 v = *reinterpret_cast<const uint4*>(turn + r * kTurn + (piece ^ (r & 7)) * 16);
        if (wave * 32 + r < rows) {
          const int2 th = out_row(r);
          *reinterpret_cast<uint4*>(fr.a.out + (int64_t)th.x * fr.a.ld_out + (int64_t)th.y * D +
                                    piece * 8) = v;
        }
      }
    } else {
      constexpr int kPasses = D * 4 / kTurn > 0 ? D * 4 / kTurn : 1;
      constexpr int kRow = D / kPasses;            // values of a row in a pass, half per g
      constexpr int kPieces32 = kRow / 4;
      static_assert(kRow * 4 <= kTurn && OB % kPasses == 0, "a pass fits");
#pragma unroll
      for (int y = 0; y < kPasses; ++y) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int b = 0; b < OB / kPasses; ++b)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x16& v = o[y * (OB / kPasses) + b];
            const int piece = g * (kPieces32 / 2) + 4 * b + i / 4;
            *reinterpret_cast<float4*>(turn + n * kTurn + (piece ^ (n & 7)) * 16) =
                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int x = 0; x < 32 * kPieces32 / 64; ++x) {
          const int r = (x * 64 + lane) / kPieces32, piece = (x * 64 + lane) % kPieces32;
          const float4 v =
              *reinterpret_cast<const float4*>(turn + r * kTurn + (piece ^ (r & 7)) * 16);
          if (wave * 32 + r < rows) {
            const int2 th = out_row(r);
            float* po = to.whole ? parts.whole_o + ((int64_t)th.x * fr.a.Hq + th.y) * D
                                 : parts.o + (int64_t)(to.slot * R + wave * 32 + r) * D;
            const int half = piece / (kPieces32 / 2), in = piece % (kPieces32 / 2);
            *reinterpret_cast<float4*>(po + half * (D / 2) + y * (kRow / 2) + 4 * in) = v;
          }
        }
      }
    }
    note_item<kPrefix, kJoin>(parts, to, q, row0, rows, at.h, wg);
    at.pos += k1 - at.k;
    at.k = 0;
    if (++at.h == a.Hk) {
      at.h = 0;
      ++at.m;
    }
  }
}

// ---- joining the parts ------------------------------------------------------------
// Part j of a result whose first part is row f of ml / o: the first workgroup
// left it in its odd slot, the ones behind it in their even slots.
__device__ __forceinline__ int64_t part_row(int64_t f, int j, int R) {
  return j == 0 ? f : f + (int64_t)(2 * j - 1) * R;
}

__device__ __forceinline__ float wave_fmax(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = __builtin_fmaxf(x, __shfl_xor(x, d));
  return x;
}

// largest of the parts' m over a wave
__device__ __forceinline__ float parts_max(const float* ml, int64_t f, int np, int R) {
  float m = FP8_NEG_INF;
  for (int j = threadIdx.x & 63; j < np; j += 64)
    m = __builtin_fmaxf(m, ml[part_row(f, j, R) * 2]);
  return wave_fmax(m);
}

template <int D>
struct Sum {
  float l, o[D / 64];          // lane i: values i D/64 ..
};

template <int D>
__device__ __forceinline__ void add_row(Sum<D>& s, const float* ml, const float* o, int64_t row,
                                        float base) {
  const int lane = threadIdx.x & 63;
  const float f = __builtin_amdgcn_exp2f(ml[row * 2] - base);
  s.l = __builtin_fmaf(ml[row * 2 + 1], f, s.l);
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    s.o[i] = __builtin_fmaf(o[row * D + lane * (D / 64) + i], f, s.o[i]);
}

// kTogether: parts whose loads go out together
template <int D, int kTogether>
__device__ __forceinline__ void add_parts(Sum<D>& s, const float* ml, const float* o, int64_t f,
                                          int np, int R, float base, int j0, int step) {
  for (int j = j0; j < np; j += kTogether * step) {
    float f_[kTogether], l_[kTogether], o_[kTogether][D / 64];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const bool is = j + u * step < np;
      const int64_t row = part_row(f, is ? j + u * step : j, R);
      f_[u] = is ? ml[row * 2] : FP8_NEG_INF;
      l_[u] = ml[row * 2 + 1];
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        o_[u][i] = o[row * D + (threadIdx.x & 63) * (D / 64) + i];
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const float w = __builtin_amdgcn_exp2f(f_[u] - base);
      if (j + u * step >= np) break;
      s.l = __builtin_fmaf(l_[u], w, s.l);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) s.o[i] = __builtin_fmaf(o_[u][i], w, s.o[i]);
    }
  }
}

template <int D>
__device__ __forceinline__ void write_row(const AttentionArgs& a, const Sum<D>& s, float base,
                                          float v_scale, int64_t token, int head) {
  const int lane = threadIdx.x & 63;
  const float inv = s.l == 0.0f ? 0.0f : v_scale / s.l;
  uint16_t* p = a.out + token * a.ld_out + (int64_t)head * D + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; i += 2) {
    const uint32_t w = pack_bf16(s.o[i] * inv, s.o[i + 1 < D / 64 ? i + 1 : i] * inv);
    if (D == 64) p[0] = (uint16_t)w;
    else *reinterpret_cast<uint32_t*>(p + i) = w;
  }
  if (a.lse && lane == 0) a.lse[token * a.Hq + head] = (base + __builtin_log2f(s.l)) * kLn2;
}

// Items that shares cut: the blocks (w, y) join the rows of the item that starts
// in workgroup w's share.  With many parts the four waves of a block share a row's
// parts.  With few, 16 lanes take a row, so that a wave has the loads of four rows
// in flight: the time is that of the chain of loads (descriptor, m, O), and with
// one row per wave the join of a prefill's 512 parts (84 MB) took 19 us longer.
constexpr int kFewParts = 8;

template <int D>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionArgs a, Parts parts,
                                                                  int R) {
  __shared__ float s_l[4], s_o[4][D];
  const Split sp = parts.split[blockIdx.x];
  if (sp.parts == 0) return;
  const float v_scale = a.v_scale[0];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t f0 = ((int64_t)2 * blockIdx.x + 1) * R;
  if (sp.parts <= kFewParts) {
    const int c = lane & 15;                       // values 4 c .. 4 c + 3 of each 64
    for (int r0 = (blockIdx.y * 4 + wave) * 4; r0 < sp.rows; r0 += gridDim.y * 16) {
      const int row = r0 + (lane >> 4);
      if (row >= sp.rows) continue;
      float2 ml[kFewParts];
      float m = FP8_NEG_INF;
#pragma unroll
      for (int j = 0; j < kFewParts; ++j)
        if (j < sp.parts)
          ml[j] = *reinterpret_cast<const float2*>(parts.ml + part_row(f0 + row, j, R) * 2);
#pragma unroll
      for (int j = 0; j < kFewParts; ++j)
        if (j < sp.parts) m = __builtin_fmaxf(m, ml[j].x);
      const float base = base_of(m);
      float l = 0.0f;
      float4 o[D / 64];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < kFewParts; ++j)
        if (j < sp.parts) {
          const float w = __builtin_amdgcn_exp2f(ml[j].x - base);
          l = __builtin_fmaf(ml[j].y, w, l);
          const float* p = parts.o + part_row(f0 + row, j, R) * D + 4 * c;
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(p + 64 * i);
            o[i].x = __builtin_fmaf(x.x, w, o[i].x);
            o[i].y = __builtin_fmaf(x.y, w, o[i].y);
            o[i].z = __builtin_fmaf(x.z, w, o[i].z);
            o[i].w = __builtin_fmaf(x.w, w, o[i].w);
          }
        }
      const float inv = l == 0.0f ? 0.0f : v_scale / l;
      const int rho = sp.row0 + row, i_n = (int)div32((uint32_t)rho, a.inv_G);
      const int64_t token = sp.token0 + i_n;
      const int head = sp.head * a.G + rho - i_n * a.G;
      uint16_t* out = a.out + token * a.ld_out + (int64_t)head * D + 4 * c;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<uint2*>(out + 64 * i) = make_uint2(pack_bf16(o[i].x * inv, o[i].y * inv),
                                                             pack_bf16(o[i].z * inv, o[i].w * inv));
      if (a.lse && c == 0) a.lse[token * a.Hq + head] = (base + __builtin_log2f(l)) * kLn2;
    }
    return;
  }
  for (int row = blockIdx.y; row < sp.rows; row += gridDim.y) {
    const float base = base_of(parts_max(parts.ml, f0 + row, sp.parts, R));
    Sum<D> s = {};
    add_parts<D, 16>(s, parts.ml, parts.o, f0 + row, sp.parts, R, base, wave, 4);
    __syncthreads();
    if (lane == 0) s_l[wave] = s.l;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s_o[wave][lane * (D / 64) + i] = s.o[i];
    __syncthreads();
    if (wave != 0) continue;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      s.l += s_l[w];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) s.o[i] += s_o[w][lane * (D / 64) + i];
    }
    const int rho = sp.row0 + row, i = (int)div32((uint32_t)rho, a.inv_G);
    write_row<D>(a, s, base, v_scale, sp.token0 + i, sp.head * a.G + rho - i * a.G);
  }
}

// Shared prefix: a wave joins a row's parts of the prefix and of its request.  The
// grid ends at kMostJoinBlocks (a dispatch holds fewer than 2^32 work-items), behind
// which a wave takes several rows.
constexpr int64_t kMostJoinBlocks = (int64_t)1 << 20;

template <int D>
__global__ __launch_bounds__(kThreads) void attention_prefix_join_kernel(AttentionArgs a, Parts p1,
                                                                         int R1, Parts p2,
                                                                         int R2) {
  for (int64_t flat = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); flat < (int64_t)a.T * a.Hq;
       flat += (int64_t)gridDim.x * 4) {
    const int2 w1 = p1.where[flat], w2 = p2.where[flat];
    if (w2.y < 0) continue;                        // a row of no request
    const float v_scale = a.v_scale[0];
    const float m1 = w1.y ? parts_max(p1.ml, w1.x, w1.y, R1) : p1.whole_ml[flat * 2];
    const float m2 = w2.y ? parts_max(p2.ml, w2.x, w2.y, R2) : p2.whole_ml[flat * 2];
    const float base = base_of(__builtin_fmaxf(m1, m2));
    Sum<D> s = {};
    if (w1.y) add_parts<D, 8>(s, p1.ml, p1.o, w1.x, w1.y, R1, base, 0, 1);
    else add_row<D>(s, p1.whole_ml, p1.whole_o, flat, base);
    if (w2.y) add_parts<D, 2>(s, p2.ml, p2.o, w2.x, w2.y, R2, base, 0, 1);
    else add_row<D>(s, p2.whole_ml, p2.whole_o, flat, base);
    const int64_t token = flat / a.Hq;
    write_row<D>(a, s, base, v_scale, token, (int)(flat - token * a.Hq));
  }
}

// ---- host ---------------------------------------------------------------------------
int compute_units() {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
      return 256;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Whether B requests' T query tokens take the 256-row tiles: from 48 rows per
// request on average, as the host does not know their lengths.  Measured on batches
// of one kind (us, 16-row against 256-row tiles): 64 requests of 2048 keys, D = 128,
// Hk = 8: 64 / 147 at 16 rows, 110 / 143 at 32, 151 / 144 at 48, 199 / 142 at 64; 4
// requests of 16000: 73 / 92 at 32, 108 / 105 at 64; 32 requests of 2048, D = 64:
// 38 / 50 at 32, 69 / 52 at 64.  A shared prefix is one request of all rows: of 32768
// keys, 59 / 64 at 48 rows, 103 / 64 at 96.
// D = 256 has the 16-row tiles only: 32 rows of O and Q fill a wave's registers
// there, and 256-row tiles that spill took 1336 us where these take 199 (32
// requests of 256 rows, 2048 keys); two 16-row blocks per wave spilled too (202,
// and 47 in place of 34 for 32 rows).
bool many_rows(int64_t T, int64_t B, int64_t G, int64_t D) { return D < 256 && T * G > 48 * B; }

struct Shape {
  bool tiles;                   // large row tiles
  int wgs, R;
};

Shape shape_of(bool tiles, int64_t D) {
  const int cus = compute_units();
  Shape s;
  s.tiles = tiles;
  s.R = tiles ? kTileWaves * 32 : kRowsD;
  s.wgs = tiles ? cus : (D == 256 ? cus : 2 * cus);
  return s;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Lays a launch's parts out at ws + at (ws may be null) and moves `at` behind.
Parts lay_out(uint8_t* ws, size_t& at, const Shape& s, int64_t D, int64_t rows_joined) {
  Parts p = {};
  auto take = [&](size_t bytes) {
    uint8_t* x = ws ? ws + at : nullptr;
    at = align256(at + bytes);
    return x;
  };
  const size_t rows = (size_t)2 * s.wgs * s.R;
  p.ml = (float*)take(rows * 2 * sizeof(float));
  p.o = (float*)take(rows * D * sizeof(float));
  if (rows_joined > 0) {
    p.where = (int2*)take(rows_joined * sizeof(int2));
    p.whole_ml = (float*)take(rows_joined * 2 * sizeof(float));
    p.whole_o = (float*)take(rows_joined * D * sizeof(float));
  } else {
    p.split = (Split*)take(s.wgs * sizeof(Split));
  }
  return p;
}

template <int D, bool kPrefix, bool kJoin>
void launch_main(const AttentionArgs& a, const Parts& p, const Shape& s, hipStream_t st) {
  const KernelArgs k = {a, p};
  if constexpr (D < 256)
    if (s.tiles) {
      hipLaunchKernelGGL((attention_tile_kernel<D, kPrefix, kJoin>), dim3(s.wgs),
                         dim3(kTileWaves * 64), 0, st, k);
      return;
    }
  if (a.page % 4 == 0)
    hipLaunchKernelGGL((attention_rows_kernel<D, kPrefix, kJoin, true>), dim3(s.wgs),
                       dim3(kThreads), 0, st, k);
  else
    hipLaunchKernelGGL((attention_rows_kernel<D, kPrefix, kJoin, false>), dim3(s.wgs),
                       dim3(kThreads), 0, st, k);
}

template <int D>
hipError_t launch_d(const AttentionArgs& a, hipStream_t st) {
  size_t at = 0;
  if (!a.prefix_len) {
    const Shape s = shape_of(many_rows(a.T, a.B, a.G, D), D);
    const Parts p = lay_out(a.ws, at, s, D, 0);
    launch_main<D, false, false>(a, p, s, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attention_join_kernel<D>, dim3(s.wgs, s.tiles ? 8 : 4), dim3(kThreads), 0,
                       st, a, p, s.R);
    return hipGetLastError();
  }
  const int64_t rows = (int64_t)a.T * a.Hq;
  const Shape s1 = shape_of(many_rows(a.T, 1, a.G, D), D);
  const Shape s2 = shape_of(many_rows(a.T, a.B, a.G, D), D);
  Parts p1 = lay_out(a.ws, at, s1, D, rows), p2 = lay_out(a.ws, at, s2, D, rows);
  p1.reset = p2.where;
  launch_main<D, true, true>(a, p1, s1, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_main<D, false, true>(a, p2, s2, st);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t blocks = (rows + 3) / 4 < kMostJoinBlocks ? (rows + 3) / 4 : kMostJoinBlocks;
  hipLaunchKernelGGL(attention_prefix_join_kernel<D>, dim3((uint32_t)blocks), dim3(kThreads), 0, st,
                     a, p1, s1.R, p2, s2.R);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(bool prefix, int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D) {
  const int64_t G = Hq / Hk;
  size_t at = 0;
  if (!prefix) {
    lay_out(nullptr, at, shape_of(many_rows(T, B, G, D), D), D, 0);
  } else {
    lay_out(nullptr, at, shape_of(many_rows(T, 1, G, D), D), D, T * Hq);
    lay_out(nullptr, at, shape_of(many_rows(T, B, G, D), D), D, T * Hq);
  }
  return at;
}

hipError_t launch_attention(const AttentionArgs& a, int D, hipStream_t st) {
  switch (D) {
    case 64: return launch_d<64>(a, st);
    case 128: return launch_d<128>(a, st);
    default: return launch_d<256>(a, st);
  }
}

}  // namespace fp8k
