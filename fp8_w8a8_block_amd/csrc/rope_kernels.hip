// Norm and rotation of queries and keys with the FP8 cache store, for gfx950.
//
// Per head x of D values: y = x * rsqrt(mean(x^2) + eps) * w, then each pair
// (a, b) of the first rot values turns by its position's angle:
// (a c - b s, b c + a s).  Queries go out in bf16; keys and values go into the
// paged cache as E4M3(y / scale) ("FP8 Quantization", D.4), so the keys are
// rounded once, from fp32, and no bf16 copy of them is written and read again.
//
// A head is held by L = D / 8 lanes (rounded up to a power of two) of 8 values
// each, one 16-byte load; the mean is a butterfly over the L lanes, and the
// rotation's partner (D / 2 away) sits in another lane of the same head, or in
// the lane itself when pairs are neighbours.  The kernel streams: a lane group
// takes `per` heads of one token, all loads of up to 4 heads issued together,
// and reads the token's angles once for them.
#include "attention_launch.h"
#include "device_common.h"
#include "launch.h"

namespace fp8k {

namespace {

constexpr int kUnroll = 4;

__device__ __forceinline__ uint32_t bf16_rne(float f) {
  return f != f ? 0x7fc0u : f32_to_bf16_rne(f);
}

// L lanes per head; per heads (of Hq + 2 Hk) per lane group and pass.
template <int L, bool kInterleaved>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRopeArgs a, int32_t per,
                                                        int32_t chunks) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int c = threadIdx.x % L;                    // this lane's 8 values of the head
  const int64_t t = item / chunks;
  if (t >= a.T) return;                             // whole lane groups leave together
  const int h0 = (int)(item - t * chunks) * per;
  const int heads = a.Hq + 2 * a.Hk;
  const int h1 = h0 + per < heads ? h0 + per : heads;
  const int64_t pos = a.positions[t], slot = a.slots[t];
  if (pos < 0 || pos >= a.max_pos) return;
  const bool keep = slot >= 0 && slot < a.capacity;
  const bool live = c * 8 < a.D;
  const bool turns = c * 8 < a.rot;
  const int half = a.rot / 2;

  // cosines and sines of this lane's values, the sine with the sign of its term
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
  }
  if (turns) {
    const float* row = a.cos_sin + pos * a.rot;
    if (kInterleaved) {
      const float4 vc = *reinterpret_cast<const float4*>(row + c * 4);
      const float4 vs = *reinterpret_cast<const float4*>(row + half + c * 4);
      const float fc[4] = {vc.x, vc.y, vc.z, vc.w}, fs[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = fc[e / 2];
        sn[e] = (e & 1) ? fs[e / 2] : -fs[e / 2];
      }
    } else {
      const bool low = c * 8 < half;
      const int j = low ? c * 8 : c * 8 - half;
      const float sign = low ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 vc = *reinterpret_cast<const float4*>(row + j + e);
        const float4 vs = *reinterpret_cast<const float4*>(row + half + j + e);
        cs[e] = vc.x; cs[e + 1] = vc.y; cs[e + 2] = vc.z; cs[e + 3] = vc.w;
        sn[e] = sign * vs.x; sn[e + 1] = sign * vs.y;
        sn[e + 2] = sign * vs.z; sn[e + 3] = sign * vs.w;
      }
    }
  }
  // lane of the rotation's other half (itself where nothing turns)
  const int partner = !turns ? c : c * 8 < half ? c + half / 8 : c - half / 8;
  const int lane_base = (threadIdx.x & 63) - c;

  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (live) {
    wq = *reinterpret_cast<const uint4*>(a.qw + c * 8);
    wk = *reinterpret_cast<const uint4*>(a.kw + c * 8);
  }
  const float k_scale = a.k_scale[0];
  const StaticDivisor vd = make_static_divisor(a.v_scale[0]);
  const float inv_d = 1.0f / (float)a.D;

  for (int h = h0; h < h1; h += kUnroll) {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u;
      x[u] = make_uint4(0, 0, 0, 0);
      if (hh < h1 && live) {
        const uint16_t* p = hh < a.Hq          ? a.q + t * a.ld_q + (int64_t)hh * a.D
                            : hh < a.Hq + a.Hk ? a.k + t * a.ld_k + (int64_t)(hh - a.Hq) * a.D
                                               : a.v + t * a.ld_v +
                                                     (int64_t)(hh - a.Hq - a.Hk) * a.D;
        x[u] = *reinterpret_cast<const uint4*>(p + c * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u;
      if (hh >= h1) break;
      if (hh >= a.Hq + a.Hk) {                      // a value head: stored as it is
        if (keep && live) {
          const int64_t off = (slot * a.Hk + (hh - a.Hq - a.Hk)) * a.D + c * 8;
          *reinterpret_cast<uint2*>(a.vc + off) = quant8_static(x[u], vd);
        }
        continue;
      }
      const bool is_q = hh < a.Hq;
      const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      const uint4 w = is_q ? wq : wk;
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      float y[8], ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = (e & 1) ? bf16_hi(xw[e / 2]) : bf16_lo(xw[e / 2]);
        ss = __builtin_fmaf(y[e], y[e], ss);
      }
#pragma unroll
      for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m);
      const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = y[e] * r * ((e & 1) ? bf16_hi(ww[e / 2]) : bf16_lo(ww[e / 2]));
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // the pair's other value: next to it, or in the partner's lane
        const float o = kInterleaved ? y[e ^ 1] : __shfl(y[e], lane_base + partner);
        z[e] = turns ? __builtin_fmaf(o, sn[e], y[e] * cs[e]) : y[e];
      }
      if (!live) continue;
      if (is_q) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = bf16_rne(z[2 * e]) | (bf16_rne(z[2 * e + 1]) << 16);
        *reinterpret_cast<uint4*>(a.q_out + t * a.ld_qo + (int64_t)hh * a.D + c * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
      } else if (keep) {
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e / 4] |= (uint32_t)e4m3_encode_one(z[e] / k_scale) << (8 * (e & 3));
        const int64_t off = (slot * a.Hk + (hh - a.Hq)) * a.D + c * 8;
        *reinterpret_cast<uint2*>(a.kc + off) = make_uint2(o[0], o[1]);
      }
    }
  }
}

int lanes_of(int64_t D) {
  int l = 2;
  while (l * 8 < D) l *= 2;
  return l;
}

// Heads per lane group: one while the step is small (latency: every head of
// every token at once), more when there are tokens enough to fill the card,
// so that a token's angles are read for several heads.
int heads_per_group(int64_t T, int heads, int L) {
  const int64_t lanes = T * heads * L;
  for (int per = 8; per > 1; per /= 2)
    if (lanes / per >= (int64_t)256 * 2048) return per;
  return 1;
}

template <int L>
void launch_l(const NormRopeArgs& a, bool inter, hipStream_t st) {
  const int heads = a.Hq + 2 * a.Hk;
  const int per = heads_per_group(a.T, heads, L);
  const int chunks = (heads + per - 1) / per;
  const int64_t items = a.T * chunks * L;
  const dim3 grid((uint32_t)((items + 255) / 256));
  if (inter)
    hipLaunchKernelGGL((norm_rope_kernel<L, true>), grid, dim3(256), 0, st, a, per, chunks);
  else
    hipLaunchKernelGGL((norm_rope_kernel<L, false>), grid, dim3(256), 0, st, a, per, chunks);
}

}  // namespace

uint64_t norm_rope_items(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
  const int L = lanes_of(D);
  const int heads = (int)(Hq + 2 * Hk), per = heads_per_group(T, heads, L);
  return ((uint64_t)T * ((heads + per - 1) / per) * L + 255) / 256 * 256;
}

hipError_t launch_norm_rope(const NormRopeArgs& a, bool interleaved, hipStream_t st) {
  switch (lanes_of(a.D)) {
    case 2: launch_l<2>(a, interleaved, st); break;
    case 4: launch_l<4>(a, interleaved, st); break;
    case 8: launch_l<8>(a, interleaved, st); break;
    case 16: launch_l<16>(a, interleaved, st); break;
    case 32: launch_l<32>(a, interleaved, st); break;
    default: launch_l<64>(a, interleaved, st); break;
  }
  return hipGetLastError();
}

}  // namespace fp8k
