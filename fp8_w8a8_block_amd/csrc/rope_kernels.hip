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
// takes several heads of one token, reads the token's angles once for them and
// has the next head's load in flight while it works on one.  8191 tokens of 32
// + 8 + 8 heads of 128 (189 MB) take 42 us, 4.5 TB/s, where a large copy moves
// 4.85; more loads in flight per lane (2, 4, 8 heads) cost occupancy and time
// (44, 47, 65 us).  With positions on three axes they take 45.1 us where the one-axis
// call takes 40.7: two more positions and four more reads of angles per lane group.
#include "attention_launch.h"
#include "device_common.h"
#include "launch.h"

namespace fp8k {

namespace {

// L lanes per head.  `chunks` lane groups share a token's Hq + 2 Hk heads: group
// j takes heads j, j + chunks, ..., so that a wave's groups read neighbouring
// heads and are mostly all at queries, at keys or at values.
// kAxes: positions on several axes.  Lane c reads the angles of pairs 4 c .. 4 c + 3
// at every axis' position, 16 bytes each, keeps each pair's axis', and hands them to
// the lanes that turn these pairs.  All reads are on their way together: with a
// branch for each axis 8191 tokens of 48 heads of 128 took 57 us, without 48 (and 45
// with twelve heads per group).
template <int L, bool kInterleaved, bool kAxes>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRopeArgs a, uint32_t chunks) {
  const uint32_t item = blockIdx.x * (256u / L) + threadIdx.x / L;
  const int c = threadIdx.x % L;                    // this lane's 8 values of the head
  const uint32_t t32 = item / chunks;
  if (t32 >= a.T) return;                           // whole lane groups leave together
  const int64_t t = t32;
  const int heads = a.Hq + 2 * a.Hk;
  const int h0 = (int)(item - t32 * chunks);
  const bool live = c * 8 < a.D;

  auto fetch = [&](int h) {
    const uint16_t* p = h < a.Hq          ? a.q + t * a.ld_q + (int64_t)h * a.D
                        : h < a.Hq + a.Hk ? a.k + t * a.ld_k + (int64_t)(h - a.Hq) * a.D
                                          : a.v + t * a.ld_v + (int64_t)(h - a.Hq - a.Hk) * a.D;
    return h < heads && live ? *reinterpret_cast<const uint4*>(p + c * 8)
                             : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 next = fetch(h0);                           // on its way while the angles are found
  const int64_t pos = a.positions[t], slot = a.slots[t];
  int64_t at[4] = {pos, pos, pos, pos};
  bool inside = pos >= 0 && pos < a.max_pos;
  if (kAxes) {
    // the last axis again for those that are not there: no branch between the loads
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      at[i] = a.positions[(int64_t)(i < a.axes ? i : a.axes - 1) * a.ld_pos + t];
      inside &= at[i] >= 0 && at[i] < a.max_pos;
    }
  }
  if (!inside) return;
  const bool keep = slot >= 0 && slot < a.capacity;
  const bool turns = c * 8 < a.rot;
  const int half = a.rot / 2;

  // cosines and sines of this lane's values, the sine with the sign of its term
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
  }
  if (kAxes) {
    // The axes of the lane's pairs, two bits each.  Each word goes through a scalar
    // register: the compiler makes an index by lane of a plain selection, and that
    // is a vector load of the launch's arguments, which lie in host memory.
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < (L + 3) / 4; ++i) {
      uint32_t w = a.axis_bits[i];
      asm("" : "+s"(w));
      word = (c >> 2) == i ? w : word;
    }
    const uint32_t bits = word >> ((c & 3) * 8);
    float vc[4] = {1.0f, 1.0f, 1.0f, 1.0f}, vs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turns) {                                    // a table of no columns holds nothing
      float4 rc[4], rs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* row = a.cos_sin + at[i] * a.rot + c * 4;
        rc[i] = *reinterpret_cast<const float4*>(row);
        rs[i] = *reinterpret_cast<const float4*>(row + half);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ci[4] = {rc[i].x, rc[i].y, rc[i].z, rc[i].w};
        const float si[4] = {rs[i].x, rs[i].y, rs[i].z, rs[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool its = (bits >> (2 * e) & 3u) == (uint32_t)i;
          vc[e] = its ? ci[e] : vc[e];
          vs[e] = its ? si[e] : vs[e];
        }
      }
    }
    const bool low = c * 8 < half;
    const int from = (threadIdx.x & 63) - c + (low ? c * 2 : c * 2 - half / 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (kInterleaved) {
        cs[e] = vc[e / 2];
        sn[e] = (e & 1) ? vs[e / 2] : -vs[e / 2];
      } else {
        const float oc = __shfl(vc[e & 3], from + e / 4), os = __shfl(vs[e & 3], from + e / 4);
        cs[e] = turns ? oc : 1.0f;
        sn[e] = !turns ? 0.0f : low ? -os : os;
      }
    }
  } else if (turns) {
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
  const int partner_lane = (threadIdx.x & 63) - c + partner;

  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (live) {
    wq = *reinterpret_cast<const uint4*>(a.qw + c * 8);
    wk = *reinterpret_cast<const uint4*>(a.kw + c * 8);
  }
  const StaticDivisor kd = make_static_divisor(a.k_scale[0]);
  const StaticDivisor vd = make_static_divisor(a.v_scale[0]);
  const float inv_d = 1.0f / (float)a.D;
  const float least = a.eps < 0x1p-100f ? 0x1p-80f : 0.0f;   // smaller sums may have lost squares

  for (int h = h0; h < heads; h += (int)chunks) {
    const uint4 x = next;
    next = fetch(h + (int)chunks);
    if (h >= a.Hq + a.Hk) {                         // a value head: stored as it is
      if (keep && live)
        *reinterpret_cast<uint2*>(a.vc + (slot * a.Hk + (h - a.Hq - a.Hk)) * a.D + c * 8) =
            quant8_static(x, vd);
      continue;
    }
    const bool is_q = h < a.Hq;
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
    const uint4 w = is_q ? wq : wk;
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    float y[8], z[8], ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = (e & 1) ? bf16_hi(xw[e / 2]) : bf16_lo(xw[e / 2]);
      ss = __builtin_fmaf(y[e], y[e], ss);
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m);
    float r = rsqrt_of(__builtin_fmaf(ss, inv_d, a.eps));
    if (__ballot(__builtin_amdgcn_fmed3f(ss, least, 0x1p+126f) != ss)) {
      // A head of the wave has squares that leave fp32's range.  Those of f x do not; f
      // stays with small x, whose 1 / rms may be beyond it.  (The test costs 0.5 to
      // 1 %: 40.3 and 40.7 us, 44.9 and 45.1 with three axes.)
      const float f = ss > 0x1p+126f ? 0x1p-80f : ss < least ? 0x1p+90f : 1.0f;
      ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(y[e] * f, y[e] * f, ss);
#pragma unroll
      for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m);
      r = rsqrt_of(__builtin_fmaf(ss, inv_d, a.eps * f * f)) * (f > 1.0f ? 1.0f : f);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= f > 1.0f ? f : 1.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      y[e] = y[e] * r * ((e & 1) ? bf16_hi(ww[e / 2]) : bf16_lo(ww[e / 2]));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // the pair's other value: next to it, or in the partner's lane
      const float o = kInterleaved ? y[e ^ 1] : __shfl(y[e], partner_lane);
      z[e] = turns ? __builtin_fmaf(o, sn[e], y[e] * cs[e]) : y[e];
    }
    if (!live) continue;
    if (is_q)
      *reinterpret_cast<uint4*>(a.q_out + t * a.ld_qo + (int64_t)h * a.D + c * 8) =
          make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]),
                     pack_bf16(z[6], z[7]));
    else if (keep)
      *reinterpret_cast<uint2*>(a.kc + (slot * a.Hk + (h - a.Hq)) * a.D + c * 8) =
          quant8_f32(z, kd);
  }
}

int lanes_of(int64_t D) {
  int l = 2;
  while (l * 8 < D) l *= 2;
  return l;
}

// Heads per lane group: one while the step is small (latency: every head of
// every token at once), up to six while three waves per SIMD are left, so that
// a token's angles are read for several heads.  8191 tokens of 48 heads of 128
// take 50 us with 2, 42.4 with 6, 45.7 with 12.  With several axes, whose angles
// cost up to four reads and an exchange between lanes, up to twelve: 51.2 us with
// 4, 48.9 with 6, 45.2 with 12, 46.2 with 24.
int heads_per_group(int64_t T, int heads, int L, bool axes) {
  const int64_t lanes = T * heads * L;
  for (int per : {12, 6, 4, 3, 2})
    if ((per <= 6 || axes) && lanes / per >= (int64_t)256 * 4 * 3 * 64) return per;
  return 1;
}

template <int L>
void launch_l(const NormRopeArgs& a, bool inter, hipStream_t st) {
  const int heads = a.Hq + 2 * a.Hk;
  const int per = heads_per_group(a.T, heads, L, a.axes > 1);
  const int chunks = (heads + per - 1) / per;
  const int64_t items = a.T * chunks * L;
  const dim3 grid((uint32_t)((items + 255) / 256));
  if (a.axes > 0 && inter)
    hipLaunchKernelGGL((norm_rope_kernel<L, true, true>), grid, dim3(256), 0, st, a, chunks);
  else if (a.axes > 0)
    hipLaunchKernelGGL((norm_rope_kernel<L, false, true>), grid, dim3(256), 0, st, a, chunks);
  else if (inter)
    hipLaunchKernelGGL((norm_rope_kernel<L, true, false>), grid, dim3(256), 0, st, a, chunks);
  else
    hipLaunchKernelGGL((norm_rope_kernel<L, false, false>), grid, dim3(256), 0, st, a, chunks);
}

}  // namespace

// (with one axis: more axes make no more groups)
uint64_t norm_rope_items(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
  const int L = lanes_of(D);
  const int heads = (int)(Hq + 2 * Hk), per = heads_per_group(T, heads, L, false);
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
