// Log probabilities of given tokens, with rank, entropy and the k most likely
// alternatives, for gfx950.
//
// With t = (x - m) c, c = scale log2(e), m the row's maximum, over one pass:
//   S = sum 2^t,  D = sum t 2^t,
//   log p = scale (x_token - m) - ln2 log2 S,  entropy = ln2 (log2 S - D / S),
// S and D rescaled when the running maximum grows.  x - m is formed first, so
// that nothing is lost at large logits or a mask of the type's lowest value.
//
// The alternatives need no second pass over the row.  It is seen as segments of
// 128 bytes, whose maxima are kept (the softmax needs them anyway).  512 threads
// hold the maximum of some segments each; the k-th largest of these bounds
// the k-th largest logit from below, so only the segments that reach it are read
// again, and of them only the logits that reach it are ranked.
//
// Many rows are bound by HBM: 2047 rows of 128000 bf16 logits (524 MB) take 105 us,
// 5.0 TB/s.  Few are bound by the way through two launches and, in the second, four
// dependent reads with barriers between: one row 4.2 + 5.6 us, 61 rows of 100003 fp32
// logits (24 MB, 5 us at a copy's rate) 9 + 5.
#include <type_traits>

#include "device_common.h"
#include "fp8w8a8_step.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8k {

namespace {

constexpr int kThreads = 512;
constexpr int kSweep = kThreads / 8;         // segments that the workgroup reads at once
constexpr int kMaxSegments = 4096;           // kept in LDS by the one-launch form
constexpr int kMaxListed = 192;              // segments read again
constexpr int kMaxRanked = 512;              // logits ranked

constexpr float kInf = __builtin_huge_valf();
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

// maximum, S, D and the number of logits above the token's, of a part of a row
struct Stats {
  float m, s, d;
  uint32_t above;
};

__device__ __forceinline__ float anchor(float m) { return m == -kInf ? 0.0f : m; }

// (x - from) pre, in fp32's range where the difference is not
__device__ __forceinline__ float apart(float x, float from, const LogprobScale& u) {
  return __builtin_fmaf(x, u.pre, -from * u.pre);
}

// What turns differences of logits into exponents.  kFar: a scale so small that
// differences beyond fp32 have a weight, or so large that scale log2(e) is beyond it;
// else c is that, and pre and post are left out (2 % of the time of a few rows).
template <bool kFar>
struct Unit {
  LogprobScale u;

  // (x - from) scale log2(e)
  __device__ __forceinline__ float exponent(float x, float from) const {
    return kFar ? apart(x, from, u) * u.c * u.post : (x - from) * u.c;
  }
  // The same for many x, a product less with `post`: (x post - from post) c.  Where from 2
  // may be beyond fp32, too, a difference is 0 or 2^-24 and more, of weight 0 with any c
  // of that size.
  struct From {
    float from, pre, lift, c;
    __device__ __forceinline__ float exponent(float x) const {
      return kFar ? __builtin_fmaf(x, pre, lift) * c : (x - from) * c;
    }
  };
  __device__ __forceinline__ From relative_to(float from) const {
    if (!kFar) return {from, 1.0f, 0.0f, u.c};
    const bool far = u.post != 1.0f && __builtin_fabsf(from) >= 1.0f;
    const float pre = far ? 1.0f : u.pre * u.post;
    return {from, pre, -from * pre, far ? 0x1.fffffep+127f : u.c};
  }
};

// (s, d) relative to the maximum m, moved to the maximum to >= m.  A NaN in s or d
// stays one, so nothing here may be 0 times infinity, nor drop a factor of 0.
template <bool kFar>
__device__ __forceinline__ void rebase(float m, float to, Unit<kFar> c, float& s, float& d) {
  const float by = m == -kInf ? 0.0f : __builtin_fmaxf(c.exponent(m, to), -1000.0f);
  const float f = __builtin_amdgcn_exp2f(by);
  d = f * __builtin_fmaf(s, by, d);
  s = f * s;
}

template <bool kFar>
__device__ __forceinline__ void join(Stats& a, float m, float s, float d, Unit<kFar> c) {
  const float to = __builtin_fmaxf(a.m, m);
  rebase(a.m, to, c, a.s, a.d);
  rebase(m, to, c, s, d);
  a.m = to;
  a.s += s;
  a.d += d;
}

// f over the wave's 64 values, in every lane
template <typename F>
__device__ __forceinline__ float wave_fold(float v, F f) {
  auto other = [](float x, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v = f(v, other(v, std::integral_constant<int, 0x128>()));     // the row of 16 turned by 8, 4, 2, 1
  v = f(v, other(v, std::integral_constant<int, 0x124>()));
  v = f(v, other(v, std::integral_constant<int, 0x122>()));
  v = f(v, other(v, std::integral_constant<int, 0x121>()));
  auto row = [&](int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
  };
  return f(f(row(0), row(16)), f(row(32), row(48)));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_fold(v, [](float a, float b) { return a + b; });
}

// the wave's sums, in every lane (above is not touched)
template <bool kFar>
__device__ __forceinline__ void join_wave(Stats& a, Unit<kFar> c) {
  const float m = wave_fold(a.m, [](float x, float y) { return __builtin_fmaxf(x, y); });
  rebase(a.m, m, c, a.s, a.d);
  a.m = m;
  a.s = wave_sum(a.s);
  a.d = wave_sum(a.d);
}

// A row as vectors of 16 bytes from the 128-byte line on in which it starts:
// vector v, value e is logit v V + e - lead.
template <bool kF32>
struct Row {
  static constexpr int V = kF32 ? 4 : 8;
  const uint4* base;
  uint32_t lead, n;            // n logits

  __device__ __forceinline__ Row(const void* logits, int64_t ld, int64_t row, int64_t vocab) {
    const uintptr_t p = (uintptr_t)logits + (uintptr_t)(row * ld) * (kF32 ? 4 : 2);
    base = reinterpret_cast<const uint4*>(p & ~(uintptr_t)127);
    lead = (uint32_t)((p & 127) / (kF32 ? 4 : 2));
    n = (uint32_t)vocab;
  }
  __device__ __forceinline__ bool whole(uint32_t v) const {
    return v * V >= lead && v * V + V <= lead + n;
  }
  __device__ __forceinline__ static void unpack(const uint4 r, float x[V]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < V; ++e)
      x[e] = kF32 ? __uint_as_float(w[e]) : (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
  // logit i < n
  __device__ __forceinline__ float at(uint32_t i) const {
    if (kF32) return reinterpret_cast<const float*>(base)[lead + i];
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[lead + i] << 16);
  }
  // any vector: -inf where there is no logit; `fits` has a bit for each that is one
  __device__ __forceinline__ uint32_t load(uint32_t v, float x[V]) const {
    if (whole(v)) {
      unpack(base[v], x);
      return (1u << V) - 1u;
    }
    uint32_t fits = 0u;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t i = v * V + e - lead;          // wraps in front of the row
      x[e] = -kInf;
      if (i < n) {
        x[e] = at(i);
        fits |= 1u << e;
      }
    }
    return fits;
  }
};

// maximum over the 8 lanes that hold a segment
__device__ __forceinline__ float segment_max(float v) {
  auto other = [](float x, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v = __builtin_fmaxf(v, other(v, std::integral_constant<int, 0xb1>()));    // lane ^ 1
  v = __builtin_fmaxf(v, other(v, std::integral_constant<int, 0x4e>()));    // lane ^ 2
  return __builtin_fmaxf(v, other(v, std::integral_constant<int, 0x141>())); // 7 - lane of 8
}

// One batch of U vectors a thread, kThreads apart: x is theirs.  `segments` of the
// batch are the part's.
template <bool kF32, int U, bool kFar>
__device__ __forceinline__ void take(const float (&x)[U][Row<kF32>::V], Unit<kFar> c, float mine,
                                     Stats& a, float* maxima, uint32_t segments) {
  constexpr int V = Row<kF32>::V;
  float top[U], m = a.m;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    top[u] = x[u][0];
#pragma unroll
    for (int e = 1; e < V; ++e) top[u] = __builtin_fmaxf(top[u], x[u][e]);
    m = __builtin_fmaxf(m, top[u]);
  }
  rebase(a.m, m, c, a.s, a.d);
  a.m = m;
  const auto from = c.relative_to(anchor(m));
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float t = from.exponent(x[u][e]), w = __builtin_amdgcn_exp2f(t);
      a.s += w;
      // a weight of 0 has an exponent of -inf, and no part in D
      a.d = __builtin_fmaf(w, __builtin_fmaxf(t, -1000.0f), a.d);
      a.above += (uint32_t)__builtin_popcountll(__ballot(x[u][e] > mine));
    }
    const float seg = segment_max(top[u]);
    const uint32_t at = u * kSweep + (threadIdx.x >> 3);
    if ((threadIdx.x & 7u) == 0 && at < segments) maxima[at] = seg;
  }
}

// A batch that may reach beyond the row or the part: every load is on its way before
// any is looked at, the vectors at the ends of the row (and there is none but those
// if it is short) are read value by value.
template <bool kF32, int U>
__device__ __forceinline__ void load_batch(const Row<kF32>& row, uint32_t seg, uint4 (&r)[U]) {
  constexpr int V = Row<kF32>::V;
  const uint32_t lo = (row.lead + V - 1) / V, hi = (row.lead + row.n) / V;    // whole: lo .. hi - 1
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t v = seg * 8u + threadIdx.x + u * kThreads;
    v = v < lo ? lo : v;
    v = v < hi ? v : hi - 1;
    r[u] = lo < hi ? row.base[v] : make_uint4(0u, 0u, 0u, 0u);
  }
}
template <bool kF32, int U, bool kFar>
__device__ __forceinline__ void take_edge(const Row<kF32>& row, const uint4 (&r)[U], uint32_t seg,
                                          uint32_t last, Unit<kFar> c, float mine, Stats& a,
                                          float* maxima) {
  constexpr int V = Row<kF32>::V;
  const uint32_t lo = (row.lead + V - 1) / V, hi = (row.lead + row.n) / V, end = last * 8u;
  float x[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t v = seg * 8u + threadIdx.x + u * kThreads;
    row.unpack(r[u], x[u]);
    if (v < lo || v >= hi || v >= end) {
      if (v < end) {
        row.load(v, x[u]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[u][e] = -kInf;
      }
    }
  }
  take<kF32, U>(x, c, mine, a, maxima, last - seg);
}

// Segments first .. last - 1 of a row, their maxima to maxima[0 ..]; the sums of
// the whole workgroup in every thread.  get_mine reads the token's logit, once the
// first loads of the row are on their way.
template <bool kF32, bool kFar, typename F>
__device__ Stats stream(const Row<kF32>& row, uint32_t first, uint32_t last, Unit<kFar> c,
                        float& mine, float* maxima, F get_mine) {
  constexpr int V = Row<kF32>::V, U = 4;
  __shared__ Stats shared[kThreads / 64];
  Stats a = {-kInf, 0.0f, 0.0f, 0u};
  mine = kInf;
  for (uint32_t seg = first; seg < last; seg += U * kSweep) {
    float* to = maxima + (seg - first);
    // all of the batch inside the row and the part, for all threads alike
    if (seg + U * kSweep <= last && row.whole(seg * 8u) &&
        row.whole((seg + U * kSweep) * 8u - 1u)) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = row.base[seg * 8u + threadIdx.x + u * kThreads];
      if (seg == first) mine = get_mine();
      float x[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) row.unpack(r[u], x[u]);
      take<kF32, U>(x, c, mine, a, to, U * kSweep);
    } else if (last - seg > 2 * kSweep) {
      uint4 r[U];
      load_batch<kF32, U>(row, seg, r);
      if (seg == first) mine = get_mine();
      take_edge<kF32, U>(row, r, seg, last, c, mine, a, to);
    } else {
      uint4 r[2];
      load_batch<kF32, 2>(row, seg, r);
      if (seg == first) mine = get_mine();
      take_edge<kF32, 2>(row, r, seg, last, c, mine, a, to);
    }
  }
  join_wave(a, c);
  if ((threadIdx.x & 63u) == 0) shared[threadIdx.x >> 6] = a;
  __syncthreads();
  Stats all = shared[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) {
    join(all, shared[w].m, shared[w].s, shared[w].d, c);
    all.above += shared[w].above;
  }
  return all;
}

// fp32 bits in the values' order
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// a logit and its place as one number: of equal logits the lower index is the larger
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
  return (uint64_t)order_key(x) << 32 | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

struct Select {
  uint64_t key[kMaxRanked];
  float super[kThreads];
  uint32_t listed[kMaxListed];
  uint32_t hist[256];
  uint32_t wave[kThreads / 64];
  uint32_t segments, ranked, bin, left;
  float bound, mine;
  Stats all;
};

// Largest key that at least k of the wave's 64 N values reach (or one between it and
// the next lower value that exactly k reach), k <= 64 N.
template <int N>
__device__ __forceinline__ uint32_t kth_key(const float (&v)[N], uint32_t k) {
  uint32_t key[N], found = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = order_key(v[i]);
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = found | (1u << bit);
    uint32_t n = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) n += (uint32_t)__builtin_popcountll(__ballot(key[i] >= t));
    if (n >= k) found = t;
    if (n == k) break;
  }
  return found;
}

// f(segment, its maximum) for every segment of a row, eight reads a thread on their way
// together: one after the other they cost the second launch 1.8 of 6.9 us (3126 segments).
template <typename F>
__device__ __forceinline__ void each_segment(const float* maxima, uint32_t segments, F f) {
  constexpr uint32_t U = 8;
  for (uint32_t s0 = threadIdx.x; s0 < segments; s0 += U * kThreads) {
    float v[U];
#pragma unroll
    for (uint32_t i = 0; i < U; ++i) {
      const uint32_t s = s0 + i * kThreads;
      v[i] = maxima[s < segments ? s : segments - 1u];
    }
#pragma unroll
    for (uint32_t i = 0; i < U; ++i)
      if (s0 + i * kThreads < segments) f(s0 + i * kThreads, v[i]);
  }
}

// Step 1 of the selection: sh.bound, which k logits at least reach.  Thread t holds the
// maximum of segments t, t + 512, ... (neighbouring ones apart, so that a cluster
// of likely tokens does not share a maximum); the k-th largest of these maxima is a
// bound, and for k up to 32 that of 64 of them, at a third of the time: it lets 24
// logits pass for k = 20 where 512 let 20 pass.  `aside` is done by the second wave
// meanwhile.  Ends with a barrier.
template <typename F>
__device__ __forceinline__ void bound_top(const float* maxima, uint32_t segments, uint32_t k,
                                          Select& sh, F aside) {
  const uint32_t tid = threadIdx.x;
  float m = -kInf;
  each_segment(maxima, segments, [&](uint32_t, float v) { m = __builtin_fmaxf(m, v); });
  sh.super[tid] = m;
  if (tid == 0) sh.segments = sh.ranked = 0u;
  __syncthreads();
  if (tid < 64) {
    float v[kThreads / 64], one[1] = {-kInf};
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) {
      v[i] = sh.super[i * 64 + tid];
      one[0] = __builtin_fmaxf(one[0], v[i]);
    }
    const float f = key_value(k <= 32 ? kth_key(one, k) : kth_key(v, k));
    if (tid == 0) sh.bound = f == f ? f : -kInf;    // below -inf in the order: no bound
  } else if (tid < 128) {
    aside();
  }
  __syncthreads();
}

// f(value, index) for every logit of the row, in any order
template <bool kF32, typename F>
__device__ __forceinline__ void each_logit(const Row<kF32>& row, F f) {
  constexpr int V = Row<kF32>::V;
  const uint32_t vectors = (row.lead + row.n + V - 1) / V;
  for (uint32_t v = threadIdx.x; v < vectors; v += kThreads) {
    float x[V];
    const uint32_t fits = row.load(v, x);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (fits >> e & 1u) f(x[e], v * V + e - row.lead);
  }
}

// Step 2: the k most likely logits of a row, by falling value and rising index.
// `log_p` turns a logit into what is written.
template <bool kF32, typename F>
__device__ void select_top(const Row<kF32>& row, const float* maxima, uint32_t segments, uint32_t k,
                           float* top, int32_t* ids, Select& sh, F log_p) {
  constexpr int V = Row<kF32>::V;
  const uint32_t tid = threadIdx.x;
  const float bound = sh.bound;
  // masked logits are not listed: the lowest of them are filled in below
  auto passes = [&](float x) { return x >= bound && x > -kInf; };
  each_segment(maxima, segments, [&](uint32_t s, float v) {
    if (!passes(v)) return;
    const uint32_t i = atomicAdd(&sh.segments, 1u);
    if (i < kMaxListed) sh.listed[i] = s;
  });
  __syncthreads();
  const uint32_t listed = sh.segments;
  auto rank_this = [&](float x, uint32_t index) {
    const uint32_t i = atomicAdd(&sh.ranked, 1u);
    if (i < kMaxRanked) sh.key[i] = rank_key(x, index);
  };
  if (listed <= kMaxListed) {
    for (uint32_t i = tid >> 3; i < listed; i += kSweep) {
      const uint32_t v = sh.listed[i] * 8u + (tid & 7u);
      float x[V];
      const uint32_t fits = row.load(v, x);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if ((fits >> e & 1u) && passes(x[e])) rank_this(x[e], v * V + e - row.lead);
    }
  }
  __syncthreads();
  uint32_t ranked = sh.ranked, equal = order_key(-kInf);
  if (listed > kMaxListed || ranked > kMaxRanked) {
    // Many equal logits, or many large ones in a few segments: the k-th largest
    // key is found digit by digit over the whole row; what is larger is ranked,
    // and the first of its equals are filled in.
    uint32_t prefix = 0u, left = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) sh.hist[tid] = 0u;
      __syncthreads();
      each_logit(row, [&](float x, uint32_t) {
        const uint32_t key = order_key(x);
        if (shift < 24 && (key >> (shift + 8)) != (prefix >> (shift + 8))) return;
        // lanes of the first one's digit count together
        const uint32_t bin = key >> shift & 255u, lead_bin = __builtin_amdgcn_readfirstlane(bin);
        const uint64_t same = __ballot(bin == lead_bin);
        if (bin != lead_bin)
          atomicAdd(&sh.hist[bin], 1u);
        else if ((tid & 63u) == (uint32_t)__builtin_ctzll(same))
          atomicAdd(&sh.hist[bin], (uint32_t)__builtin_popcountll(same));
      });
      __syncthreads();
      if (tid < 64) {
        // lane l: digits 255 - 4 l .. 252 - 4 l
        uint32_t h[4], sum = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += h[i] = sh.hist[255u - 4u * tid - i];
        uint32_t before = sum;
        for (int i = 1; i < 64; i <<= 1) {
          const uint32_t o = __shfl_up(before, i);
          if ((int)tid >= i) before += o;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < left && left <= before + h[i]) {
            sh.bin = 255u - 4u * tid - i;
            sh.left = left - before;
          }
          before += h[i];
        }
      }
      __syncthreads();
      prefix |= sh.bin << shift;
      left = sh.left;
    }
    equal = prefix;
    if (tid == 0) sh.ranked = 0u;
    __syncthreads();
    each_logit(row, [&](float x, uint32_t index) {
      if (order_key(x) > equal) rank_this(x, index);
    });
    __syncthreads();
    ranked = sh.ranked;                             // k - left
  }
  // eight at a time, so that their reads overlap: LDS beyond the last holds what it may
  if (tid < ranked) {
    const uint64_t mine = sh.key[tid];
    uint32_t rank = 0u;
    for (uint32_t j = 0; j < ranked; j += 8u)
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) rank += j + e < ranked && sh.key[j + e] > mine;
    if (rank < k) {
      top[rank] = log_p(key_value((uint32_t)(mine >> 32)));
      ids[rank] = (int32_t)(0xffffffffu - (uint32_t)mine);
    }
  }
  // the first logits of key `equal`, by index
  uint32_t filled = ranked;
  const uint32_t vectors = (row.lead + row.n + V - 1) / V;
  for (uint32_t v0 = 0; filled < k && v0 < vectors; v0 += kThreads) {
    float x[V];
    uint32_t fits = v0 + tid < vectors ? row.load(v0 + tid, x) : 0u;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if ((fits >> e & 1u) && order_key(x[e]) != equal) fits &= ~(1u << e);
    const uint32_t own = (uint32_t)__builtin_popcount(fits);
    uint32_t upto = own;
    for (int i = 1; i < 64; i <<= 1) {
      const uint32_t o = __shfl_up(upto, i);
      if ((int)(tid & 63u) >= i) upto += o;
    }
    __syncthreads();
    if ((tid & 63u) == 63u) sh.wave[tid >> 6] = upto;
    __syncthreads();
    uint32_t place = filled + upto - own;
    for (uint32_t w = 0; w < kThreads / 64; ++w) {
      if (w < (tid >> 6)) place += sh.wave[w];
      filled += sh.wave[w];
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (fits >> e & 1u) {
        if (place < k) {
          top[place] = log_p(x[e]);
          ids[place] = (int32_t)((v0 + tid) * V + e - row.lead);
        }
        ++place;
      }
  }
}

// A row's outputs.  Its sums are sh.all and its token's logit sh.mine once `sums` has been
// called by the second wave.
template <bool kF32, typename F>
__device__ void finish(const LogprobArgs& a, int64_t t, const Row<kF32>& row,
                       const float* maxima, uint32_t segments, Select& sh, F sums) {
  bound_top(maxima, segments, a.k ? (uint32_t)a.k : 1u, sh, sums);
  const Stats all = sh.all;
  const bool none = all.m == -kInf && all.s == 0.0f;   // nothing but -inf
  const bool good = none || all.s == all.s;            // no NaN, no +inf
  const float from = anchor(all.m), log_s = __builtin_amdgcn_logf(all.s);
  const float nan = __builtin_nanf("");
  auto log_p = [&](float x) {
    return !good        ? nan
           : x == -kInf ? -kInf
                        : __builtin_fmaf(apart(x, from, a.unit), a.unit.z, -log_s * kLn2);
  };
  if (threadIdx.x == 0) {
    const bool given = a.tokens[t] >= 0 && a.tokens[t] < a.V;
    a.logprobs[t] = given ? log_p(sh.mine) : 0.0f;
    a.ranks[t] = given && good ? (int32_t)all.above : -1;
    a.entropy[t] = !good ? nan : none ? 0.0f : (log_s - all.d / all.s) * kLn2;
    a.lse[t] = !good ? nan : none ? -kInf : __builtin_fmaf(log_s, kLn2, all.m * a.scale);
  }
  if (a.k == 0) return;
  float* top = a.top + t * a.k;
  int32_t* ids = a.ids + t * a.k;
  if (good) {
    select_top(row, maxima, segments, (uint32_t)a.k, top, ids, sh, log_p);
  } else if (threadIdx.x < (uint32_t)a.k) {
    top[threadIdx.x] = nan;
    ids[threadIdx.x] = -1;
  }
}

// the logit of the row's token; +inf, which nothing is above, if there is none
template <bool kF32>
__device__ __forceinline__ float token_logit(const LogprobArgs& a, int64_t t, const Row<kF32>& row) {
  const int64_t token = a.tokens[t];
  return token >= 0 && token < a.V ? row.at((uint32_t)token) : kInf;
}

__device__ __forceinline__ uint32_t segments_of(uint32_t lead, int64_t vocab, int per) {
  return (lead + (uint32_t)vocab + per - 1u) / per;
}

// One workgroup per row: the pass and the selection.
template <bool kF32, bool kFar>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a) {
  extern __shared__ float maxima[];
  __shared__ Select sh;
  const int64_t t = blockIdx.x;
  const Row<kF32> row(a.logits, a.ld, t, a.V);
  const Unit<kFar> c = {a.unit};
  float mine;
  const uint32_t segments = segments_of(row.lead, a.V, 8 * Row<kF32>::V);
  const Stats all = stream(row, 0u, segments, c, mine, maxima,
                           [&] { return token_logit(a, t, row); });
  finish(a, t, row, maxima, segments, sh, [&] {
    if (threadIdx.x == 64) {
      sh.all = all;
      sh.mine = mine;
    }
  });
}

// Few rows: the pass over `parts` parts of each, every one of `share` segments, ...
template <bool kF32, bool kFar>
__global__ __launch_bounds__(kThreads) void logprob_part_kernel(LogprobArgs a, uint32_t parts,
                                                                uint32_t share) {
  const int64_t t = blockIdx.x / parts;
  const uint32_t p = blockIdx.x - (uint32_t)t * parts;
  const Row<kF32> row(a.logits, a.ld, t, a.V);
  const Unit<kFar> c = {a.unit};
  float mine;
  const uint32_t segments = segments_of(row.lead, a.V, 8 * Row<kF32>::V);
  const uint32_t first = p * share < segments ? p * share : segments;
  const uint32_t last = first + share < segments ? first + share : segments;
  Stats* stats = reinterpret_cast<Stats*>(a.ws);
  float* maxima = reinterpret_cast<float*>(stats + (uint64_t)a.T * parts) +
                  (uint64_t)blockIdx.x * share;
  const Stats all = stream(row, first, last, c, mine, maxima,
                           [&] { return token_logit(a, t, row); });
  if (threadIdx.x == 0) stats[blockIdx.x] = all;
}

// ... and what follows from them.
template <bool kF32, bool kFar>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs a, uint32_t parts,
                                                                uint32_t share) {
  __shared__ Select sh;
  const int64_t t = blockIdx.x;
  const Row<kF32> row(a.logits, a.ld, t, a.V);
  const Unit<kFar> c = {a.unit};
  const Stats* stats = reinterpret_cast<const Stats*>(a.ws) + (uint64_t)t * parts;
  // on their way while the bound is found: the token and the first of the parts' sums
  const int64_t token = a.tokens[t];
  const uint32_t lane = threadIdx.x & 63u;
  const Stats near = stats[lane < parts ? lane : 0u];
  const float* maxima = reinterpret_cast<const float*>(reinterpret_cast<const Stats*>(a.ws) +
                                                       (uint64_t)a.T * parts) +
                        (uint64_t)t * parts * share;
  finish(a, t, row, maxima, segments_of(row.lead, a.V, 8 * Row<kF32>::V), sh, [&] {
    const float mine = token >= 0 && token < a.V ? row.at((uint32_t)token) : kInf;
    Stats all = {-kInf, 0.0f, 0.0f, 0u};
    if (lane < parts) all = near;
    for (uint32_t p = lane + 64u; p < parts; p += 64u) {
      join(all, stats[p].m, stats[p].s, stats[p].d, c);
      all.above += stats[p].above;
    }
    for (int i = 1; i < 64; i <<= 1) all.above += __shfl_xor(all.above, i);
    join_wave(all, c);
    if (threadIdx.x == 64) {
      sh.all = all;
      sh.mine = mine;
    }
  });
}

struct Plan {
  uint32_t parts, share;        // parts of a row, segments of a part
};

// One workgroup per row, whose segment maxima LDS holds, for a row of up to 16 sweeps
// or a row for each compute unit; else parts of two sweeps, or of whole batches of
// four, about 1024 in all.  Times in us: V 32000 fp32 (16 sweeps) 8.3 whole and 8.4 in
// parts of two for 1 row, 8.8 and 10.0 for 61, bf16 (8 sweeps) 7.8 and 8.4, 8.7 and
// 9.4; V 128000 bf16 (32 sweeps) 18.3 and 10.0 for 1 row, 19.8 and 13.8 for 61, 21.3
// whole and 17.6 in parts of four for 128, 22.6 and 25.1 for 256, 55.7 and 68.2 for
// 1023; fp32 29.6 and 33.6 for 256, 67.6 and 64.6 for 600, 95.0 and 103.1 for 1023.
Plan plan_of(bool f32, int64_t T, int64_t V) {
  // the row may start anywhere in its first segment
  const int64_t per = f32 ? 32 : 64, segments = (V + 2 * per - 2) / per;
  const int64_t sweeps = (segments + kSweep - 1) / kSweep;
  int64_t each = (sweeps * T + 1023) / 1024;
  each = each <= 2 ? 2 : (each + 3) / 4 * 4;
  if (T >= 256 || sweeps <= 16 || each >= sweeps) each = sweeps;
  if (each > kMaxSegments / kSweep) each = kMaxSegments / kSweep;
  const int64_t share = each * kSweep;
  return {(uint32_t)((segments + share - 1) / share), (uint32_t)share};
}

}  // namespace

size_t logprobs_workspace(bool f32, int64_t T, int64_t V, int64_t k) {
  (void)k;
  const Plan p = plan_of(f32, T, V);
  if (p.parts == 1) return 0;
  const uint64_t items = (uint64_t)T * p.parts;
  return items * sizeof(Stats) + items * p.share * sizeof(float);
}

uint64_t logprobs_items(bool f32, int64_t T, int64_t V, int64_t k) {
  (void)k;
  return (uint64_t)T * plan_of(f32, T, V).parts * kThreads;
}

template <bool kF32, bool kFar>
static hipError_t launch(const LogprobArgs& a, hipStream_t st) {
  const Plan p = plan_of(kF32, a.T, a.V);
  if (p.parts == 1) {
    hipLaunchKernelGGL((logprob_kernel<kF32, kFar>), dim3((uint32_t)a.T), dim3(kThreads),
                       p.share * sizeof(float), st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((logprob_part_kernel<kF32, kFar>), dim3((uint32_t)(a.T * p.parts)),
                     dim3(kThreads), 0, st, a, p.parts, p.share);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((logprob_join_kernel<kF32, kFar>), dim3((uint32_t)a.T), dim3(kThreads), 0,
                     st, a, p.parts, p.share);
  return hipGetLastError();
}

hipError_t launch_logprobs(LogprobArgs a, bool f32, hipStream_t st) {
  // from 2^-100 on a difference beyond fp32 has a weight of 0, as its infinity does
  const bool far = a.scale < 0x1p-100f || a.scale >= 0x1p+126f;
  a.unit.pre = a.scale < 1.0f ? 0.5f : 1.0f;
  a.unit.post = a.scale >= 0x1p+126f ? 2.0f : 1.0f;
  a.unit.z = a.scale / a.unit.pre;
  a.unit.c = (far ? a.unit.z / a.unit.post : a.scale) * kLog2e;
  if (far) return f32 ? launch<true, true>(a, st) : launch<false, true>(a, st);
  return f32 ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace fp8k
