// 4-bit weights with group scales, for gfx950: packing, quantization by groups
// and the product out = x . W^T of bf16 rows with them.
//
// With w = s (c - z) for the codes c of a group,
//   out[m, n] = sum_g s[n, g] ( sum_k x[m, k] (16 + c[n, k]) - (16 + z[n, g]) sum_k x[m, k] ).
// 16 + c is a bf16 number whose lower mantissa bits are the code: a shift and
// one and-or turn two codes of the packed layout into a pair of the matrix
// unit's operand.  The group's sum of x is one more column of the product, by a
// column of ones, and comes out in the lanes and registers that need it.
#include "device_common.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8k {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
  const uint4 r = make_uint4(((d << 3) & kMask) | kBase, ((d >> 1) & kMask) | kBase,
                             ((d >> 5) & kMask) | kBase, ((d >> 9) & kMask) | kBase);
  return __builtin_bit_cast(bf16x8, r);
}

// A lane reads 16 bytes of its row, 32 values: of the 128 values of a block, quarter
// q = lane / 16.  A product takes 8 values from each quarter and must stay within
// one group, so where groups are shorter than a block the quarters' dwords trade
// places: across the wave's halves for 64, and across its rows of 16, too, for 32.
// Afterwards dword j holds the values from x_offset<G>(j, q) on.
template <int G>
__device__ __forceinline__ void spread(uint32_t (&d)[4]) {
  if (G <= 64) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto r = __builtin_amdgcn_permlane32_swap(d[j], d[j + 2], false, false);
      d[j] = r[0];
      d[j + 2] = r[1];
    }
  }
  if (G == 32) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const auto r = __builtin_amdgcn_permlane16_swap(d[j], d[j + 1], false, false);
      d[j] = r[0];
      d[j + 1] = r[1];
    }
  }
}

template <int G>
__device__ __forceinline__ int x_offset(int j, int q) {
  if (G == 128) return q * 32 + j * 8;
  if (G == 64) return (j >> 1) * 64 + (q & 1) * 32 + (q >> 1) * 16 + (j & 1) * 8;
  return j * 32 + q * 8;
}

// Up to 16 MT rows of x with 16 NT rows of the weight per workgroup, whose W waves
// share K: wave w takes every W-th block of 128 values.
template <int MT, int NT, int W, int G, bool kZeros>
__global__ __launch_bounds__(64 * W) void int4_rows_kernel(Int4Args a, uint32_t m_tiles) {
  __shared__ float part[W][MT * 16][NT * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const uint32_t tile = blockIdx.x / m_tiles;
  const int64_t n0 = (int64_t)tile * (16 * NT);
  const int64_t m0 = (int64_t)(blockIdx.x - tile * m_tiles) * (16 * MT);
  const int blocks = a.K / 128;
  constexpr int GPB = 128 / G;                      // groups of a block

  // rows behind the last are read as the last and not stored
  const uint8_t* wp[NT];
  const float* sp[NT];
  const uint8_t* zp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int64_t n = n0 + 16 * t + l16;
    n = n < a.N ? n : a.N - 1;
    wp[t] = a.codes + n * (a.K / 2) + q * 16;
    sp[t] = a.scales + n * (a.K / G);
    zp[t] = kZeros ? a.zeros + n * (a.K / G) : nullptr;
  }
  const uint16_t* xp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t m = m0 + 16 * i + l16;
    m = m < a.M ? m : a.M - 1;
    xp[i] = a.x + m * a.ld_x;
  }

  const bf16x8 ones = __builtin_bit_cast(
      bf16x8, make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u));
  f32x4 acc[MT][NT] = {};
  for (int b = wave; b < blocks; b += W) {
    uint32_t d[NT][4];
    float s[NT][GPB], z[NT][GPB];
    bf16x8 x[MT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 v = *reinterpret_cast<const uint4*>(wp[t] + (int64_t)b * 64);
      d[t][0] = v.x;
      d[t][1] = v.y;
      d[t][2] = v.z;
      d[t][3] = v.w;
#pragma unroll
      for (int g = 0; g < GPB; ++g) {
        s[t][g] = sp[t][b * GPB + g];
        z[t][g] = 16.0f + (kZeros ? (float)zp[t][b * GPB + g] : 8.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[i][j] = *reinterpret_cast<const bf16x8*>(xp[i] + (int64_t)b * 128 + x_offset<G>(j, q));
#pragma unroll
    for (int t = 0; t < NT; ++t) spread<G>(d[t]);
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      constexpr int J = 4 / GPB;                    // products of a group
      f32x4 sum[MT] = {}, p[MT][NT] = {};
#pragma unroll
      for (int j = g * J; j < (g + 1) * J; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
          sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i][j], ones, sum[i], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8 w = operand(d[t][j]);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            p[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i][j], w, p[i][t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][t][r] = __builtin_fmaf(
                s[t][g], __builtin_fmaf(-z[t][g], sum[i][r], p[i][t][r]), acc[i][t][r]);
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][16 * i + 4 * q + r][16 * t + l16] = acc[i][t][r];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * NT * 256; e += 64 * W) {
    const int m = e / (16 * NT), n = e % (16 * NT);
    float v = part[0][m][n];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][m][n];
    if (m0 + m < a.M && n0 + n < a.N)
      a.out[(m0 + m) * a.ld_out + n0 + n] = (uint16_t)pack_bf16(v, v);
  }
}

struct RowsPlan {
  int mt, nt;
};

RowsPlan rows_plan(int64_t M, int64_t N) {
  const int mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int nt = N >= 64 * 1024 || mt == 4 ? 4 : N >= 16 * 1024 || mt == 2 ? 2 : 1;
  return {mt, nt};
}

uint64_t rows_grid(int64_t M, int64_t N) {
  const RowsPlan p = rows_plan(M, N);
  return (uint64_t)((N + 16 * p.nt - 1) / (16 * p.nt)) * (uint64_t)((M + 16 * p.mt - 1) / (16 * p.mt));
}

template <int MT, int NT, int W>
void launch_rows(const Int4Args& a, int group, hipStream_t st) {
  const uint32_t m_tiles = (uint32_t)((a.M + 16 * MT - 1) / (16 * MT));
  const dim3 grid((uint32_t)rows_grid(a.M, a.N)), block(64 * W);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a, m_tiles); };
  switch (group * 2 + (a.zeros != nullptr)) {
    case 64: go(int4_rows_kernel<MT, NT, W, 32, false>); break;
    case 65: go(int4_rows_kernel<MT, NT, W, 32, true>); break;
    case 128: go(int4_rows_kernel<MT, NT, W, 64, false>); break;
    case 129: go(int4_rows_kernel<MT, NT, W, 64, true>); break;
    case 256: go(int4_rows_kernel<MT, NT, W, 128, false>); break;
    default: go(int4_rows_kernel<MT, NT, W, 128, true>); break;
  }
}

}  // namespace

uint64_t int4_linear_items(int64_t M, int64_t N, int64_t K) {
  (void)K;
  return rows_grid(M, N) * 512u;
}

hipError_t launch_int4_linear(const Int4Args& a, int group, hipStream_t st) {
  const RowsPlan p = rows_plan(a.M, a.N);
  switch (p.mt * 8 + p.nt) {
    case 9: launch_rows<1, 1, 8>(a, group, st); break;
    case 10: launch_rows<1, 2, 8>(a, group, st); break;
    case 12: launch_rows<1, 4, 8>(a, group, st); break;
    case 18: launch_rows<2, 2, 8>(a, group, st); break;
    case 20: launch_rows<2, 4, 4>(a, group, st); break;
    default: launch_rows<4, 4, 4>(a, group, st); break;
  }
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
