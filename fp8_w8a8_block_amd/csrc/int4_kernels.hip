// 4-bit weights with group scales, for gfx950: packing, quantization by groups
// and the product out = x . W^T of bf16 rows with them.
//
// With w = s (c - z) for the codes c of a group,
//   out[m, n] = sum_g s[n, g] ( sum_k x[m, k] (16 + c[n, k]) - (16 + z[n, g]) sum_k x[m, k] ).
// 16 + c is a bf16 number whose lower mantissa bits are the code: a shift and
// one and-or turn two codes of the packed layout into a pair of the matrix
// unit's operand.  The products of a group are exact and its sums fp32, so the
// scale is applied once per group and result, not rounded into the weight.
//
// Few rows are bound by the weight's bytes: K / 2 a row and 4 or 5 for each group.
// 13 rows with 128000 x 4096 (groups of 128, zero points; 287 MB) take 64.9 us, 4.4
// TB/s of the 4.9 that a copy reaches; one row with 4096 x 4096 (8.9 MB) 4.2 us and
// with 4096 x 14336 (groups of 64, zero points; 34 MB) 9.9, of which about 3 are the
// launch and the first loads' way.  Many rows are bound by what a group costs
// besides its products: 1000 rows with 11008 x 4096 take 109 us on a constant input
// and 121 on random ones, for which the clock falls from 2.4 to about 2 GHz;
// the matrix unit is busy for 38% of the cycles, the vector unit for 59% (unpacking,
// the groups' scaling, x's way to LDS), LDS for 56%; with zero points they take 132.
// Quantizing a weight of 11008 x 4096 takes 38 us (3.0 TB/s), 128000 x 4096 388 (3.4),
// packing them 16 (4.3) and 158 (5.0).
#include <type_traits>

#include "device_common.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8k {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- packing and quantization ----------------------------------------------

// 8 codes to 4 bytes: the even values' in the lower half word, the odd ones' in the upper
__device__ __forceinline__ uint32_t pack8(const uint32_t v[8]) {
  uint32_t d = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) d |= v[e] << (16 * (e & 1) + 4 * (e / 2));
  return d;
}

__global__ __launch_bounds__(256) void int4_pack_kernel(const uint8_t* __restrict__ values,
                                                        int64_t ld_v, uint8_t* __restrict__ codes,
                                                        uint32_t chunks, uint64_t total) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < total;
       i += (uint64_t)gridDim.x * 256u) {
    const uint64_t n = i / chunks;
    const uint2 b = *reinterpret_cast<const uint2*>(values + n * ld_v + (i - n * chunks) * 8u);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ((e < 4 ? b.x : b.y) >> (8 * (e & 3))) & 15u;
    reinterpret_cast<uint32_t*>(codes)[i] = pack8(v);
  }
}

// One lane per 8 values, G / 8 neighbouring lanes per group.  total and the grid's
// stride are multiples of 16, so the lanes of a group stay together.
template <int G>
__global__ __launch_bounds__(256) void int4_quant_kernel(
    const uint16_t* __restrict__ w, int64_t ld_w, uint8_t* __restrict__ codes,
    float* __restrict__ scales, uint8_t* __restrict__ zeros, uint32_t chunks, uint64_t total) {
  constexpr int L = G / 8;
  for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < total;
       i += (uint64_t)gridDim.x * 256u) {
    const uint64_t n = i / chunks;
    const uint4 p = *reinterpret_cast<const uint4*>(w + n * ld_w + (i - n * chunks) * 8u);
    const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
    float x[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = (e & 1) ? bf16_hi(pw[e / 2]) : bf16_lo(pw[e / 2]);
      lo = __builtin_fminf(lo, x[e]);
      hi = __builtin_fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1) {
      lo = __builtin_fminf(lo, __shfl_xor(lo, m));
      hi = __builtin_fmaxf(hi, __shfl_xor(hi, m));
    }
    const float s = zeros ? (hi - lo) / 15.0f : __builtin_fmaxf(-lo, hi) / 7.0f;
    float z = zeros ? 0.0f : 8.0f;
    if (zeros && s > 0.0f) z = __builtin_fminf(__builtin_rintf(-lo / s), 15.0f);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = s > 0.0f ? __builtin_rintf(x[e] / s) + z : z;
      v[e] = (uint32_t)__builtin_amdgcn_fmed3f(c, 0.0f, 15.0f);
    }
    reinterpret_cast<uint32_t*>(codes)[i] = pack8(v);
    if ((threadIdx.x & (L - 1)) == 0) {
      scales[i / L] = s;
      if (zeros) zeros[i / L] = (uint8_t)z;
    }
  }
}

// ---- products ----------------------------------------------------------------

// A packed dword as 8 bf16 operand values 16 + c (bits of 16.0: 0x4180; the
// code's unit is mantissa bit 3)
__device__ __forceinline__ bf16x8 operand(uint32_t d) {
  constexpr uint32_t kMask = 0x00780078u;
  uint32_t base = 0x41804180u;
  asm("" : "+v"(base));                              // in a register: and and or in one
  const uint4 r = make_uint4(((d << 3) & kMask) | base, ((d >> 1) & kMask) | base,
                             ((d >> 5) & kMask) | base, ((d >> 9) & kMask) | base);
  return __builtin_bit_cast(bf16x8, r);
}

// A lane reads 16 bytes of its row, 32 values: of the 128 values of a block, quarter
// q = lane / 16.  A product takes 8 values from each quarter and must stay within
// one group, so where groups are shorter than a block the quarters' dwords trade
// places: across the wave's halves for 64, and across its rows of 16, too, for 32.
// Afterwards dword j holds the values from x_offset<S>(j, q) on.
template <int S>
__device__ __forceinline__ void spread(uint32_t (&d)[4]) {
  if (S <= 64) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto r = __builtin_amdgcn_permlane32_swap(d[j], d[j + 2], false, false);
      d[j] = r[0];
      d[j + 2] = r[1];
    }
  }
  if (S == 32) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const auto r = __builtin_amdgcn_permlane16_swap(d[j], d[j + 1], false, false);
      d[j] = r[0];
      d[j + 1] = r[1];
    }
  }
}

template <int S>
__device__ __forceinline__ int x_offset(int j, int q) {
  if (S == 128) return q * 32 + j * 8;
  if (S == 64) return (j >> 1) * 64 + (q & 1) * 32 + (q >> 1) * 16 + (j & 1) * 8;
  return j * 32 + q * 8;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void store_bf16(const Int4Args& a, int64_t m, int64_t n, float v) {
  if (m < a.M && n < a.N) a.out[m * a.ld_out + n] = (uint16_t)pack_bf16(v, v);
}

// Not finite: a sum left fp32's range on the way, or x or the weight's scales hold what is
// not finite.
__device__ __forceinline__ bool beyond(float v) { return !(__builtin_fabsf(v) < __builtin_huge_valf()); }

// out[m, n] for a result that is `beyond`, from the definition in 64 bits: x (16 + code) and
// its sums leave fp32's range from |x| = 2^112 on, where s (c - z) x need not.  All lanes of
// a wave call, 16 neighbouring ones with one m, whose row of x they search together for an
// infinity or a NaN, which makes it NaN; only those that want it get a result.
__device__ float again(const Int4Args& a, int64_t m, int64_t n, int group, bool wanted) {
  const uint16_t* x = a.x + m * a.ld_x;
  uint32_t bad = 0u;
  for (int k = (threadIdx.x & 15u) * 8; k < a.K; k += 128) {
    const u32x4 r = *reinterpret_cast<const u32x4*>(x + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) bad |= ((r[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  }
  if (__ballot(bad != 0u) >> (threadIdx.x & 48u) & 0xffffu) return __builtin_nanf("");
  if (!wanted) return 0.0f;
  const uint8_t* w = a.codes + n * (a.K / 2);
  double sum = 0.0;
#pragma unroll 1
  for (int k0 = 0; k0 < a.K; k0 += group) {
    const int64_t g = n * (a.K / group) + k0 / group;
    const int z = a.zeros ? a.zeros[g] : 8;
    double part = 0.0;
#pragma unroll 1
    for (int k = k0; k < k0 + group; k += 8) {
      const u32x4 r = *reinterpret_cast<const u32x4*>(x + k);
      const uint32_t d = *reinterpret_cast<const uint32_t*>(w + k / 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = (e & 1) ? bf16_hi(r[e / 2]) : bf16_lo(r[e / 2]);
        part += (double)v * (double)((int)(d >> (16 * (e & 1) + 4 * (e / 2)) & 15u) - z);
      }
    }
    sum += (double)a.scales[g] * part;
  }
  return (float)sum;
}

constexpr int kFewGroups = 64;  // groups of a row that LDS holds, for each of up to four waves

// Up to 4 rows of x with 16 rows of the weight.  The 16 rows of the matrix unit's
// operand are the 4 rows of x times the 4 products j of a block: row 4 m + j holds
// the values of x's row m that product j multiplies, so one load a block brings
// all of x, and product j's result is right where row = 4 m + j: in register j of
// quarter m.  Column n, quarter m of the wave is output (m, n).  The groups' sums of
// x are the same product with ones.
//
// The workgroup's waves share K: each takes a run of units of four blocks, the next
// of which is in flight while it works on one.  The matrix unit has time for the
// 16-fold product of one row (it is idle otherwise), and reading x as its operand
// spares the lanes' sum at the end.  The groups' scales go through LDS: read where they
// are used, 16 rows at 4 bytes each, they cost more requests than the codes.
template <int G, bool kZeros>
__global__ __launch_bounds__(512) void int4_few_kernel(Int4Args a) {
  constexpr int GPB = 128 / G, J = 4 / GPB;         // products of a group
  constexpr int kStage = kFewGroups / 4;            // of which a thread brings every 4 waves-th
  extern __shared__ float2 few_lds[];               // scales and offsets; then the waves' parts
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int blocks = a.K / 128, units = (blocks + 3) / 4;
  const int most = kFewGroups * (waves < 4 ? waves : 4) / (4 * GPB);  // units of a chunk of K
  // rows behind the last are read as the last and not stored
  const int rows = (int)(a.N - n0 < 16 ? a.N - n0 : 16);
  const int64_t m = (l16 >> 2) < a.M ? l16 >> 2 : a.M - 1;
  const uint8_t* w = a.codes + n0 * (a.K / 2);
  const uint32_t wo = (uint32_t)(l16 < rows ? l16 : rows - 1) * (uint32_t)(a.K / 2) + q * 16;
  const uint16_t* x = a.x + m * a.ld_x + x_offset<G>(l16 & 3, q);

  struct Unit {
    u32x4 w[4];
    bf16x8 x[4];
  };
  auto fetch = [&](Unit& u, int at) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = at * 4 + i < blocks ? at * 4 + i : blocks - 1;
      u.w[i] = *reinterpret_cast<const u32x4*>(w + (uint32_t)b * 64u + wo);
      u.x[i] = *reinterpret_cast<const bf16x8*>(x + b * 128);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const bf16x8 ones = __builtin_bit_cast(
      bf16x8, make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u));
  float acc = 0.0f;
  for (int c0 = 0; c0 < units; c0 += most) {
    const int cn = units - c0 < most ? units - c0 : most;
    const int held = (cn * 4 < blocks - c0 * 4 ? cn * 4 : blocks - c0 * 4) * GPB;
    const int pitch = held | 1;
    if (c0) __syncthreads();
    // the groups of 16 rows, neighbouring threads along a row
    float gs[kStage];
    uint32_t gz[kStage];
    const int gr = (int)__umulhi(threadIdx.x, 0xffffffffu / (uint32_t)(4 * waves) + 1u);
    const int gc = (int)threadIdx.x - gr * 4 * waves;                // threadIdx.x / (4 waves), the rest
    const float* gs0 = a.scales + n0 * (a.K / G) + c0 * 4 * GPB;
    const uint8_t* gz0 = kZeros ? a.zeros + n0 * (a.K / G) + c0 * 4 * GPB : nullptr;
    const uint32_t go = (uint32_t)(gr < rows ? gr : rows - 1) * (uint32_t)(a.K / G);
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      if (i * 4 * waves >= held) break;             // all of the workgroup
      const int g = gc + i * 4 * waves < held ? gc + i * 4 * waves : held - 1;
      gs[i] = gs0[go + (uint32_t)g];
      if (kZeros) gz[i] = gz0[go + (uint32_t)g];
    }
    __builtin_amdgcn_sched_barrier(0);
    const int first = c0 + (int)((uint32_t)cn * wave / waves);
    const int last = c0 + (int)((uint32_t)cn * (wave + 1) / waves);
    Unit here, next;
    fetch(here, first < last ? first : c0);
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int g = gc + i * 4 * waves;
      if (i * 4 * waves >= held) break;
      if (g < held)
        few_lds[gr * pitch + g] = make_float2(gs[i], 16.0f + (kZeros ? (float)gz[i] : 8.0f));
    }
    __syncthreads();
    const float2* of = few_lds + l16 * pitch;
    auto multiply = [&](const Unit& u, int at) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at * 4 + i >= blocks) break;            // all of the wave
        uint32_t d[4] = {u.w[i].x, u.w[i].y, u.w[i].z, u.w[i].w};
        spread<G>(d);
        const f32x4 zero = {}, sum = mfma(u.x[i], ones, zero);
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = mfma(u.x[i], operand(d[j]), zero)[j];
#pragma unroll
        for (int g = 0; g < GPB; ++g) {
          float v = p[g * J], o = sum[g * J];
#pragma unroll
          for (int j = 1; j < J; ++j) {
            v += p[g * J + j];
            o += sum[g * J + j];
          }
          const float2 sz = of[((at - c0) * 4 + i) * GPB + g];
          acc = __builtin_fmaf(sz.x, __builtin_fmaf(-sz.y, o, v), acc);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int at = first; at < last; at += 2) {
      fetch(next, at + 1 < last ? at + 1 : at);
      multiply(here, at);
      if (at + 1 >= last) break;
      fetch(here, at + 2 < last ? at + 2 : at);
      multiply(next, at + 1);
    }
  }

  if (waves > 1) {
    float* part = reinterpret_cast<float*>(few_lds);
    __syncthreads();
    part[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll 4
    for (int i = 1; i < waves; ++i) acc += part[i * 64 + lane];
  }
  const bool redo = beyond(acc) && q < a.M && l16 < rows;
  if (__ballot(redo)) {                             // the lanes' row of x is the one they read
    const float v = again(a, q < a.M ? q : a.M - 1, n0 + (l16 < rows ? l16 : 0), G, redo);
    acc = redo ? v : acc;
  }
  store_bf16(a, q, n0 + l16, acc);
}

// Sum of 8 bf16 values and what v holds.
__device__ __forceinline__ float sum8(u32x4 x) {
  float v = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t pair = x[e];
    v = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair),
                                        __builtin_bit_cast(bf16x2, 0x3f803f80u), v, false);
  }
  return v;
}

// Sum over the L neighbouring lanes (4, 8 or 16) of each L, in all of them.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  auto other = [](float x, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v += other(v, std::integral_constant<int, 0xb1>());               // lane ^ 1
  v += other(v, std::integral_constant<int, 0x4e>());               // lane ^ 2
  if (L >= 8) v += other(v, std::integral_constant<int, 0x141>());  // 7 - lane of 8
  if (L >= 16) v += other(v, std::integral_constant<int, 0x140>()); // 15 - lane of 16
  return v;
}

// 16 MT rows of x with 16 NT WN rows of the weight per workgroup of WN x WK waves, over
// a run of K (`runs` of them; more than one: the sums go to a.parts and are added
// by int4_join_kernel).  The waves of WK take every WK-th block of K.  x goes through
// LDS, KB blocks at a time, with its sums by groups, and so do the scales and
// offsets, kTileGroups at a time; both twice, the next while the last are in use.
// The codes come straight to the waves that multiply them, kAhead blocks ahead.
//
// 64 rows of x: a wave unpacks 32 rows of the weight for four products each.  Tried
// for 1000 rows with 11008 x 4096, 109 us: 64 rows of the weight a wave, with half the
// LDS reads, but two waves a SIMD, 116 (4096 x 8192 x 8192: 564 and 608); the next
// product's x read ahead 108.7, with zero points 594 for 564, as registers spill; rows
// of x at other distances in LDS the same; products of 32 x 32 x 16, half as many
// and with no copies of the sums, the same, too (with zero points 4% less); x's way
// to LDS spread between the products 111; an XCD's workgroups on neighbouring rows of
// the weight, which then fewer of the L2s read, 125 for 124 (random inputs; 721 for 684).
// The 64-row tiles with zero points in groups of 64 and 128 spill 5 registers, those of
// groups of 32 without them 6.
template <int MT, int NT, int WN, int WK, int G, bool kZeros>
__global__ __launch_bounds__(64 * WN * WK) __attribute__((amdgpu_waves_per_eu(MT >= 4 ? 3 : 4)))
void int4_tile_kernel(Int4Args a, uint32_t m_tiles, uint32_t runs) {
  constexpr int GPB = 128 / G, J = 4 / GPB, kThreads = 64 * WN * WK;
  constexpr int kRowsM = 16 * MT, kRowsN = 16 * NT * WN;
  constexpr int kAhead = MT >= 4 ? 2 : 4;
  constexpr int KB = MT >= 4 ? 1 : WK > 4 ? 8 : 4;                  // blocks of x in LDS
  constexpr int kTurns = KB / WK;                                   // of a wave with them
  constexpr int kPitch = KB * 128 + 8;                              // of a row of x there
  constexpr int kStage = kRowsM * KB * 16 / kThreads;               // 16-byte pieces a thread
  constexpr int kTileGroups = MT >= 4 && GPB < 4 ? 8 : 16 * WK;
  constexpr int kHeld = kTileGroups / GPB;                          // blocks whose groups LDS holds
  constexpr int kStageG = kRowsN * kTileGroups / kThreads;
  static_assert(kRowsM * KB * 16 % kThreads == 0 && kRowsN * kTileGroups % kThreads == 0 &&
                kHeld % (4 * WK) == 0 && 4 % kTurns == 0, "");
  typedef std::conditional_t<kZeros, float2, float> Group;          // scale (and offset)
  __shared__ uint16_t xs[2][kRowsM * kPitch];
  __shared__ float sums[2][KB * GPB][kRowsM];
  __shared__ Group gs[2][kRowsN * (kTileGroups + 1)];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave / WK, wk = wave % WK;
  // neighbouring workgroups take the m tiles of one n tile, then the next run
  const uint32_t run = blockIdx.x % runs, rest = blockIdx.x / runs;
  const int64_t n0 = (int64_t)(rest / m_tiles) * kRowsN;
  const int64_t m0 = (int64_t)(rest % m_tiles) * kRowsM;
  const int blocks = a.K / 128;
  const int first = (int)((uint64_t)(uint32_t)blocks * run / runs);
  const int last = (int)((uint64_t)(uint32_t)blocks * (run + 1) / runs);

  // rows of the weight behind the last are read as the last and not stored
  const int rows_n = (int)(a.N - n0 < kRowsN ? a.N - n0 : kRowsN);
  const int rows_m = (int)(a.M - m0 < kRowsM ? a.M - m0 : kRowsM);
  const uint8_t* wb = a.codes + n0 * (a.K / 2);
  uint32_t wo[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = 16 * (wn * NT + t) + l16;
    wo[t] = (uint32_t)(n < rows_n ? n : rows_n - 1) * (uint32_t)(a.K / 2) + q * 16;
  }
  auto fetch_w = [&](u32x4 (&r)[NT], int b) __attribute__((always_inline)) {
    b = b < blocks ? b : blocks - 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      r[t] = *reinterpret_cast<const u32x4*>(wb + (uint32_t)b * 64u + wo[t]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // rows of x behind the last: few rows skip them (what LDS holds in their place goes
  // into results that are not stored), many read the last again, without a branch
  constexpr bool kSkip = MT == 1;
  u32x4 stage[kStage];
  auto fetch_x = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int e = i * kThreads + threadIdx.x, r = e / (KB * 16), c = e % (KB * 16);
      const int b = b0 + c / 16 < blocks ? b0 + c / 16 : blocks - 1;
      if (kSkip && r >= rows_m) continue;
      const int64_t m = m0 + (r < rows_m ? r : rows_m - 1);
      stage[i] = *reinterpret_cast<const u32x4*>(a.x + m * a.ld_x + b * 128 + c % 16 * 8);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto keep_x = [&](int buffer) __attribute__((always_inline)) {
    constexpr int L = G / 8;                        // pieces of a group
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int e = i * kThreads + threadIdx.x, r = e / (KB * 16), c = e % (KB * 16);
      if (kSkip && r >= rows_m) continue;
      *reinterpret_cast<u32x4*>(&xs[buffer][r * kPitch + c * 8]) = stage[i];
      const float v = sum_lanes<L>(sum8(stage[i]));
      if (c % L == 0) sums[buffer][c / L][r] = kZeros ? v : v * -24.0f;
    }
  };
  float stage_s[kStageG];
  uint8_t stage_z[kStageG];
  const int per_row = a.K / G;
  const float* gs0 = a.scales + n0 * per_row;
  const uint8_t* gz0 = kZeros ? a.zeros + n0 * per_row : nullptr;
  auto fetch_g = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kStageG; ++i) {
      const int e = i * kThreads + threadIdx.x, r = e / kTileGroups, c = e % kTileGroups;
      const int g = b0 * GPB + c < per_row ? b0 * GPB + c : per_row - 1;
      const uint32_t at = (uint32_t)(r < rows_n ? r : rows_n - 1) * (uint32_t)per_row + (uint32_t)g;
      stage_s[i] = gs0[at];
      if (kZeros) stage_z[i] = gz0[at];
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto keep_g = [&](int buffer) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kStageG; ++i) {
      const int e = i * kThreads + threadIdx.x, r = e / kTileGroups, c = e % kTileGroups;
      Group& to = gs[buffer][r * (kTileGroups + 1) + c];
      if constexpr (kZeros)
        to = make_float2(stage_s[i], -16.0f - (float)stage_z[i]);
      else
        to = stage_s[i];
    }
  };
  auto read_x = [&](bf16x8 (&r)[MT], const uint16_t* xb, int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      r[i] = *reinterpret_cast<const bf16x8*>(xb + i * 16 * kPitch + x_offset<G>(k, q));
  };

  f32x4 acc[MT][NT] = {};
  u32x4 w[kAhead][NT];
  fetch_x(first);
  fetch_g(first);
#pragma unroll
  for (int j = 0; j < kAhead; ++j) fetch_w(w[j], first + j * WK + wk);
  keep_x(0);
  keep_g(0);
  fetch_x(first + KB);
  __syncthreads();
  int buffer = 0, gbuffer = 0;
  for (int b = first; b < last; b += 4 * WK) {
    const int at = (b - first) % kHeld;             // among the blocks whose groups are held
    if (at == 0) fetch_g(b + kHeld);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int mine = j * WK + wk;                 // this wave's block, counted from b
      if (b + mine < last) {
        const int held = mine % KB;                 // its place in LDS
        const uint16_t* xb = &xs[buffer][l16 * kPitch + held * 128];
        const Group* gb =
            &gs[gbuffer][(wn * NT * 16 + l16) * (kTileGroups + 1) + (at + mine) * GPB];
        uint32_t d[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          d[t][0] = w[j % kAhead][t].x;
          d[t][1] = w[j % kAhead][t].y;
          d[t][2] = w[j % kAhead][t].z;
          d[t][3] = w[j % kAhead][t].w;
          spread<G>(d[t]);
        }
        bf16x8 x[MT];
#pragma unroll
        for (int g = 0; g < GPB; ++g) {
          // the sums start at what the offsets make of the group's sum of x
          Group sz[NT];
          f32x4 p[MT][NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) sz[t] = gb[t * 16 * (kTileGroups + 1) + g];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const f32x4 sum =
                *reinterpret_cast<const f32x4*>(&sums[buffer][held * GPB + g][16 * i + 4 * q]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if constexpr (kZeros)
                p[i][t] = sum * sz[t].y;
              else
                p[i][t] = sum;
            }
          }
#pragma unroll
          for (int k = g * J; k < (g + 1) * J; ++k) {
            read_x(x, xb, k);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const bf16x8 o = operand(d[t][k]);
#pragma unroll
              for (int i = 0; i < MT; ++i) p[i][t] = mfma(x[i], o, p[i][t]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float s;
            if constexpr (kZeros)
              s = sz[t].x;
            else
              s = sz[t];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[i][t][e] = __builtin_fmaf(s, p[i][t][e], acc[i][t][e]);
              asm volatile("" : "+v"(acc[i][t]));   // here, not after the next group's products
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      fetch_w(w[j % kAhead], b + mine + kAhead * WK);
      if (j % kTurns == kTurns - 1) {               // the next blocks of x
        buffer ^= 1;
        keep_x(buffer);
        if (j == 3 && at + 4 * WK == kHeld) keep_g(gbuffer ^ 1);
        fetch_x(b + (j + 1) * WK + KB);
        __syncthreads();
      }
    }
    if (at + 4 * WK == kHeld) gbuffer ^= 1;
  }

  if constexpr (WK > 1) {
    // the waves of a tile add up their parts, in order; xs is free behind the barrier
    constexpr int kTile = MT * NT * 256;
    static_assert(WK == 1 || sizeof(xs) >= sizeof(float) * WN * WK * kTile, "");
    float* part = reinterpret_cast<float*>(xs);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<f32x4*>(&part[((wave * MT + i) * NT + t) * 256 + lane * 4]) = acc[i][t];
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int o = 1; o < WK; ++o)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[i][t] += *reinterpret_cast<const f32x4*>(
              &part[(((wave + o) * MT + i) * NT + t) * 256 + lane * 4]);
  }
  uint32_t redo = 0u;                               // a bit for each result
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + 16 * i + 4 * q + e;
        const int64_t n = n0 + 16 * (wn * NT + t) + l16;
        if (runs == 1)
          store_bf16(a, m, n, acc[i][t][e]);
        else if (m < a.M && n < a.N)
          a.parts[((int64_t)run * a.M + m) * a.N + n] = acc[i][t][e];
        if (beyond(acc[i][t][e]) && m < a.M && n < a.N) redo |= 1u << ((i * NT + t) * 4 + e);
      }
  if (runs > 1 || __ballot(redo != 0u) == 0u) return;
#pragma unroll 1
  for (int b = 0; b < MT * NT * 4; ++b) {
    const bool mine = redo >> b & 1u;
    if (__ballot(mine) == 0u) continue;
    const int64_t m = m0 + 16 * (b / (NT * 4)) + 4 * q + b % 4;
    const int64_t n = n0 + 16 * (wn * NT + b / 4 % NT) + l16;
    const float v = again(a, m < a.M ? m : a.M - 1, n, G, mine);
    if (mine) store_bf16(a, m, n, v);
  }
}

// The runs' sums, added in the order of K: a row of out per blockIdx.y.
__global__ __launch_bounds__(256) void int4_join_kernel(Int4Args a, uint32_t runs, int group) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, m = blockIdx.y;
  const int64_t total = a.M * a.N;
  const float* part = a.parts + m * a.N + n;
  f32x4 v = {};
  if (n + 4 <= a.N && a.N % 4 == 0) {
    v = *reinterpret_cast<const f32x4*>(part);
#pragma unroll 4
    for (uint32_t r = 1; r < runs; ++r) v += *reinterpret_cast<const f32x4*>(part + r * total);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= a.N) break;
      v[e] = part[e];
      for (uint32_t r = 1; r < runs; ++r) v[e] += part[r * total + e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) store_bf16(a, m, n + e, v[e]);
  uint32_t redo = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (beyond(v[e])) redo |= 1u << e;              // 0 behind the last
  if (__ballot(redo != 0u) == 0u) return;
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    const bool mine = redo >> e & 1u;
    if (__ballot(mine) == 0u) continue;
    const float r = again(a, m, n + e, group, mine);
    if (mine) store_bf16(a, m, n + e, r);
  }
}

// The kernel's tile (m 0: int4_few_kernel), its workgroups' waves, runs of K.
struct Plan {
  uint32_t m, n, waves, runs;
};

// All times in us, groups of 128, K 4096 unless another is given.
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  const int64_t blocks = K / 128, units = (blocks + 3) / 4, tiles16 = (N + 15) / 16;
  auto tiles_of = [&](int64_t m, int64_t n) { return ((M + m - 1) / m) * ((N + n - 1) / n); };
  // A card's worth of workgroups where the tiles are fewer, as the waves of one leave
  // a compute unit half idle, in runs of 8 blocks at least, of 4 while units are idle.
  auto runs_of = [&](int64_t m, int64_t n, int64_t want) {
    const int64_t tiles = tiles_of(m, n);
    int64_t runs = tiles < want ? want / tiles : 1, most = blocks / 8;
    if (tiles * most < 256) most = blocks / 4 < 256 / tiles ? blocks / 4 : 256 / tiles;
    runs = runs < most ? runs : most;
    return (uint32_t)(runs < 1 ? 1 : runs);
  };
  // Up to 4 rows: int4_few_kernel, until its reads of x, one for every 16 rows of the
  // weight, outweigh it: M 4, N 24576 13.1 against 15.0 of the 16 x 64 tiles, N 28672
  // 14.8 / 15.3, N 40000 25.0 / 22.0 (M 1: 21.2 / 21.0).
  if (M <= 4 && tiles16 <= 1792) {
    // Four waves share K while the card holds them all at once, else two, then one:
    // N 4096 4.5 with 4, 5.8 with 2, 5.2 with 8; N 11008 8.6 with 4, 8.1 with 2, 9.1
    // with 1; N 24576 14.6 with 4, 13.9 with 2, 12.2 with 1.  Eight for few tiles
    // and a long K (N 1024, K 14336: 7.7, 8.5 with 4), each of two units at least
    // (N 1024, K 4096: 4.1 with 4, 4.4 with 8).
    int64_t waves = tiles16 <= 64 ? 8 : tiles16 <= 512 ? 4 : tiles16 < 1024 ? 2 : 1;
    while (waves > 1 && units < 2 * waves) waves /= 2;
    return {0, 16, (uint32_t)waves, 1};
  }
  if (M <= 16) {
    // A workgroup for each compute unit where N allows it, and no smaller tile, as x is
    // read for each: M 16, N 4096 8.6 with 16 rows of the weight, 8.8 with 32, 10.4
    // with 64; N 5120 14.8, 8.9, 10.6; N 8192 15.8, 9.6, 10.7; N 11008 21.9, 13.3, 10.9.
    // 128 rows where x is heavy, too: N 128000, M 16 68.9 with 64, 64.4 with 128; M 5
    // 56.9 and 59.3.
    if (N > 8 * 1024) return {16, M > 8 && N >= 64 * 1024 ? 128u : 64u, 8, 1};
    // a long K is cut instead: N 4096, K 8192, M 5 / 16 11.1 / 11.9 in four runs of 64
    // rows, 11.2 / 14.5 whole in 16; K 14336 14.0 / 15.1 and 16.8 / 23.3
    if (K >= 8 * 1024) return {16, 64, 8, runs_of(16, 64, 256)};
    return {16, N > 4 * 1024 ? 32u : 16u, 8, 1};
  }
  // 32 rows of x while that is a workgroup for each compute unit at most, beyond it 64,
  // for which the codes are unpacked half as often: M 64, N 11008 18.5 with 32, 22.5
  // with 64; M 200, N 4096 18.6 / 23.4; M 100, N 11008 34.4 / 31.6; M 500, N 11008
  // 98.5 / 63.4.  The runs: M 64, N 4096 17.8 in one, 13.5 in four, 18.2 in eight; of
  // 64 rows M 300, N 4096 33.0 in one, 27.9 in three.
  if (M <= 32 || tiles_of(32, 128) <= 256) return {32, 128, 8, runs_of(32, 128, 256)};
  return {64, 128, 4, runs_of(64, 128, 512)};
}

uint64_t grid_of(const Plan& p, int64_t M, int64_t N) {
  const uint64_t m = p.m ? p.m : 4;
  return ((uint64_t)N + p.n - 1) / p.n * (((uint64_t)M + m - 1) / m) * p.runs;
}

template <typename F>
void with_groups(const Int4Args& a, int group, F f) {
  switch (group * 2 + (a.zeros != nullptr)) {
    case 64: f(std::integral_constant<int, 32>(), std::false_type()); break;
    case 65: f(std::integral_constant<int, 32>(), std::true_type()); break;
    case 128: f(std::integral_constant<int, 64>(), std::false_type()); break;
    case 129: f(std::integral_constant<int, 64>(), std::true_type()); break;
    case 256: f(std::integral_constant<int, 128>(), std::false_type()); break;
    default: f(std::integral_constant<int, 128>(), std::true_type()); break;
  }
}

template <int MT, int NT, int WN, int WK>
void launch_tile(const Int4Args& a, const Plan& p, int group, hipStream_t st) {
  const dim3 grid((uint32_t)grid_of(p, a.M, a.N));
  const uint32_t m_tiles = (uint32_t)((a.M + 16 * MT - 1) / (16 * MT));
  with_groups(a, group, [&](auto g, auto zeros) {
    hipLaunchKernelGGL(
        (int4_tile_kernel<MT, NT, WN, WK, decltype(g)::value, decltype(zeros)::value>), grid,
        dim3(64 * WN * WK), 0, st, a, m_tiles, p.runs);
  });
}

void launch_few(const Int4Args& a, const Plan& p, int group, hipStream_t st) {
  const uint32_t groups = (uint32_t)(a.K / group);
  const uint32_t most = kFewGroups * (p.waves < 4 ? p.waves : 4);
  const uint32_t held = groups < most ? groups : most;
  uint32_t lds = 16u * (held | 1u) * sizeof(float2);
  if (lds < p.waves * 256u) lds = p.waves * 256u;
  with_groups(a, group, [&](auto g, auto zeros) {
    hipLaunchKernelGGL((int4_few_kernel<decltype(g)::value, decltype(zeros)::value>),
                       dim3((uint32_t)grid_of(p, a.M, a.N)), dim3(64 * p.waves), lds, st, a);
  });
}

}  // namespace

uint64_t int4_linear_items(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_of(M, N, K);
  return grid_of(p, M, N) * 64u * p.waves;
}

size_t int4_workspace(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_of(M, N, K);
  return p.runs > 1 ? (size_t)p.runs * (size_t)M * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_int4_linear(const Int4Args& a, int group, hipStream_t st) {
  Plan p = plan_of(a.M, a.N, a.K);
  if (!a.parts) p.runs = 1;
  switch (p.m * 1024 + p.n) {
    case 16: launch_few(a, p, group, st); break;
    case 16 * 1024 + 16: launch_tile<1, 1, 1, 8>(a, p, group, st); break;
    case 16 * 1024 + 32: launch_tile<1, 1, 2, 4>(a, p, group, st); break;
    case 16 * 1024 + 64: launch_tile<1, 1, 4, 2>(a, p, group, st); break;
    case 16 * 1024 + 128: launch_tile<1, 1, 8, 1>(a, p, group, st); break;
    case 32 * 1024 + 128: launch_tile<2, 1, 8, 1>(a, p, group, st); break;
    case 64 * 1024 + 128: launch_tile<4, 2, 4, 1>(a, p, group, st); break;
    default: return hipErrorInvalidConfiguration;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.runs == 1) return e;
  hipLaunchKernelGGL(int4_join_kernel, dim3((uint32_t)((a.N + 1023) / 1024), (uint32_t)a.M),
                     dim3(256), 0, st, a, p.runs, group);
  return hipGetLastError();
}

hipError_t launch_int4_pack(const uint8_t* values, int64_t ld_v, uint8_t* codes, int64_t N,
                            int64_t K, hipStream_t st) {
  const uint64_t total = (uint64_t)N * (uint64_t)(K / 8), want = (total + 255) / 256;
  hipLaunchKernelGGL(int4_pack_kernel, dim3((uint32_t)(want < 8192 ? want : 8192)), dim3(256), 0,
                     st, values, ld_v, codes, (uint32_t)(K / 8), total);
  return hipGetLastError();
}

hipError_t launch_int4_quant(const uint16_t* w, int64_t ld_w, uint8_t* codes, float* scales,
                             uint8_t* zeros, int64_t N, int64_t K, int group, hipStream_t st) {
  const uint64_t total = (uint64_t)N * (uint64_t)(K / 8), want = (total + 255) / 256;
  const dim3 grid((uint32_t)(want < 8192 ? want : 8192));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, w, ld_w, codes, scales, zeros,
                       (uint32_t)(K / 8), total);
  };
  if (group == 32)
    go(int4_quant_kernel<32>);
  else if (group == 64)
    go(int4_quant_kernel<64>);
  else
    go(int4_quant_kernel<128>);
  return hipGetLastError();
}

}  // namespace fp8k
