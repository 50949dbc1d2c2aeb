// Residual addition, RMS norm and FP8 quantization in one pass, for gfx950.
//
//   r = bf16(x + residual),  v = r / sqrt(mean(r^2) + eps) * weight,
//   q = E4M3(v / s), s = amax / 448 over 128 values or the row, or given.
//
// HBM-bound: 6 bytes read and written per value for the stream, 1 for the code
// (2 more for a bf16 copy).  A row is held in registers as the bf16 values r,
// so it is read once; W waves share it, each lane C 16-byte chunks of it, and
// 16 neighbouring lanes hold a 128-group, whose maximum is a DPP reduction.
// 8191 rows of 4096 with codes by groups (236 MB) take 44 us, 5.4 TB/s, where a copy
// of 2 GiB moves 4.9; 2049 of 7168 with the bf16 norm and codes by rows (132 MB) 24 to
// 29 us; 4 rows 3.1 us, the way through two loads, a sum across waves and a store.
#include "device_common.h"
#include "fp8w8a8.h"
#include "step_launch.h"

namespace fp8k {

namespace {

constexpr int kNoCodes = -1;

// Sum over a row's W waves, the same in all of its lanes.  `red` is used once.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  if (W == 1) return v;
  if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) t += red[i];
  return t;
}

template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = wave_max(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) t = red[i] > t ? red[i] : t;
  return t;
}

// E4M3 codes of 8 fp32 values of a group (|z| <= its amax), as quant8.  amax is fp32
// here, not bf16: from about 2^-136 down amax / 448 is rounded to few quanta of 2^-149,
// and the quotient can reach 671.  The conversion does not saturate, so it is cut.
__device__ __forceinline__ uint2 quant8_group(const float z[8], const GroupDivisor& d) {
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = __builtin_copysignf(__builtin_fminf(quotient_abs(z[4 * h + e], d), kE4M3Max),
                                 z[4 * h + e]);
    o[h] = e4m3_pack4_mag(q[0], q[1], q[2], q[3]);
  }
  return make_uint2(o[0], o[1]);
}

// W waves per row (1: four rows to a workgroup, else one), C chunks of 8 values
// per lane, chunk c W 64 + lane.
template <int W, int C, int kMode>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_quant_kernel(NormQuantArgs a) {
  __shared__ float red_sum[W], red_again[W];
  __shared__ uint32_t red_max[W];
  const int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (t >= a.T) return;                             // W == 1 only, a whole wave
  const uint32_t lane = W == 1 ? threadIdx.x & 63u : threadIdx.x;
  const uint32_t chunks = (uint32_t)a.H / 8u;

  uint4 v[C], w[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t i = c * (64u * W) + lane;
    v[c] = i < chunks ? *reinterpret_cast<const uint4*>(a.x + t * a.ld_x + i * 8u)
                      : make_uint4(0u, 0u, 0u, 0u);
  }
  if (a.r) {
    uint4 r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * (64u * W) + lane;
      r[c] = i < chunks ? *reinterpret_cast<const uint4*>(a.r + t * a.ld_r + i * 8u)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * (64u * W) + lane;
      uint32_t p[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
      const uint32_t q[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p[e] = pack_bf16(bf16_lo(p[e]) + bf16_lo(q[e]), bf16_hi(p[e]) + bf16_hi(q[e]));
      v[c] = make_uint4(p[0], p[1], p[2], p[3]);
      if (i < chunks) *reinterpret_cast<uint4*>(a.r_out + t * a.ld_ro + i * 8u) = v[c];
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t i = c * (64u * W) + lane;
    w[c] = i < chunks ? *reinterpret_cast<const uint4*>(a.w + i * 8u) : make_uint4(0u, 0u, 0u, 0u);
  }

  // sum of (f r)^2; f, a power of two, keeps the squares of far values in range
  auto squares = [&](float f) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t p[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16_lo(p[e]) * f, hi = bf16_hi(p[e]) * f;
        ss = __builtin_fmaf(lo, lo, ss);
        ss = __builtin_fmaf(hi, hi, ss);
      }
    }
    return ss;
  };
  const float inv_h = 1.0f / (float)a.H;
  float f = 1.0f, ss = row_sum<W>(squares(1.0f), red_sum);
  if (ss > 0x1p+126f || (ss < 0x1p-80f && a.eps < 0x1p-100f)) {   // the whole row agrees
    f = ss > 1.0f ? 0x1p-80f : 0x1p+90f;
    ss = row_sum<W>(squares(f), red_again);
  }
  // v = (r up) rs weight: 1 / rms of a row that small may be beyond fp32, so f stays with r.
  // (One product more a value, under 1 % of the time of 8191 rows of 4096; a branch around
  // it, or the row made larger in its registers, spills where 16 waves hold 8 chunks a lane:
  // 104 and 77 us for 500 rows of 65536 with codes by rows, 45 like this.)
  const float up = f > 1.0f ? f : 1.0f;
  const float rs = rsqrt_of(__builtin_fmaf(ss, inv_h, a.eps * f * f)) * (f > 1.0f ? 1.0f : f);

  auto value = [&](int c, float z[8]) {
    const uint32_t p[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
    const uint32_t g[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[2 * e] = bf16_lo(p[e]) * up * rs * bf16_lo(g[e]);
      z[2 * e + 1] = bf16_hi(p[e]) * up * rs * bf16_hi(g[e]);
    }
  };
  auto absmax = [](const float z[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(z[e]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    return m;
  };
  GroupDivisor row = {};
  StaticDivisor fixed = {};
  if (kMode == FP8_SCALE_ROW) {
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float z[8];
      value(c, z);
      const uint32_t b = absmax(z);
      m = b > m ? b : m;
    }
    row = make_divisor(__uint_as_float(row_max<W>(m, red_max)));
    if (lane == 0) a.s[t * a.ld_s] = row.s;
  }
  if (kMode == FP8_SCALE_TENSOR) fixed = make_static_divisor(a.scale[0]);

#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t i = c * (64u * W) + lane;
    float z[8];
    value(c, z);
    uint2 code = make_uint2(0u, 0u);
    if (kMode == FP8_SCALE_BLOCK) {
      const GroupDivisor d = make_divisor(__uint_as_float(row16_max(absmax(z))));
      code = quant8_group(z, d);
      if (i < chunks && (lane & 15u) == 0) a.s[t * a.ld_s + i / 16u] = d.s;
    } else if (kMode == FP8_SCALE_ROW) {
      code = quant8_group(z, row);
    } else if (kMode == FP8_SCALE_TENSOR) {
      code = quant8_f32(z, fixed);
    }
    if (i >= chunks) continue;
    if (kMode != kNoCodes) *reinterpret_cast<uint2*>(a.q + t * a.ld_q + i * 8u) = code;
    if (a.y)
      *reinterpret_cast<uint4*>(a.y + t * a.ld_y + i * 8u) =
          make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]),
                     pack_bf16(z[6], z[7]));
  }
}

template <int W, int C>
void launch_wc(const NormQuantArgs& a, int mode, hipStream_t st) {
  const dim3 grid((uint32_t)(W == 1 ? (a.T + 3) / 4 : a.T)), block(W == 1 ? 256 : 64 * W);
  if (!a.q)
    hipLaunchKernelGGL((norm_quant_kernel<W, C, kNoCodes>), grid, block, 0, st, a);
  else if (mode == FP8_SCALE_BLOCK)
    hipLaunchKernelGGL((norm_quant_kernel<W, C, FP8_SCALE_BLOCK>), grid, block, 0, st, a);
  else if (mode == FP8_SCALE_ROW)
    hipLaunchKernelGGL((norm_quant_kernel<W, C, FP8_SCALE_ROW>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_quant_kernel<W, C, FP8_SCALE_TENSOR>), grid, block, 0, st, a);
}

}  // namespace

// By the width alone, so that a row's results do not depend on how many come with it.
// Times in us of 4 / 8191 rows with a residual and codes by groups: H 512 2.5 / 9.8
// with one wave, 2.6 / 14.4 with four; H 2048 2.7 / 25.1 with four of one chunk, 4.1 /
// 27.0 with one of four; H 4096 3.1 / 44.4 with eight of one, 3.4 / 44.5 with four of
// two, 6.1 / 48.2 with one of eight; H 7168 3.8 / 73.1 with eight of two, 4.4 / 75.6
// with four of four; H 16384 4.9 / 166.5 with sixteen of two, 6.8 / 164.7 with four
// of eight; H 32768 8.1 / 359 with sixteen of four, 8.4 / 357 with eight of eight.
// H 65536 13.0 / 764 (4.9 TB/s) with sixteen of eight, which spill 8 registers without
// codes (8.9 / 810) and 2 with codes by rows (11.8 / 740).
hipError_t launch_norm_quant(const NormQuantArgs& a, int mode, hipStream_t st) {
  const int chunks = a.H / 8;
  if (chunks <= 64)
    launch_wc<1, 1>(a, mode, st);
  else if (chunks <= 256)
    launch_wc<4, 1>(a, mode, st);
  else if (chunks <= 512)
    launch_wc<8, 1>(a, mode, st);
  else if (chunks <= 1024)
    launch_wc<8, 2>(a, mode, st);
  else if (chunks <= 2048)
    launch_wc<16, 2>(a, mode, st);
  else if (chunks <= 4096)
    launch_wc<16, 4>(a, mode, st);
  else
    launch_wc<16, 8>(a, mode, st);
  return hipGetLastError();
}

}  // namespace fp8k
