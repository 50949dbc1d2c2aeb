// Block tables and slot maps of one serving step, for gfx950.
//
// The paged cache stores a token at slot = block * page + offset ("Quantization
// guide for serving: FP8, AWQ, GPTQ": paged blocks).  With c_r tokens cached
// and n_r new ones, request r has ceil(c_r / p) blocks, needs
// ceil((c_r + n_r) / p), and takes the difference from the free list, behind
// what the requests before it take.  Token offsets and block offsets are both
// exclusive prefix sums over the requests.
//
// One launch: every workgroup forms the prefix sums itself, 1024 requests at a
// time (up to 4 per thread, a wave scan, a scan over the waves), and answers for its
// own stretch of tokens and its own requests' table entries.  A token of a
// block that this step hands out reads the free list, not the table entry that
// another workgroup may be writing, so no workgroup waits for another.  The
// sums cost a few microseconds of latency per 1024 requests, less than a
// second launch that would read them.  Bound by that latency and the launch's:
// 256 decoding requests take 4.9 us, 65536 tokens of 96 prompts (1 MB) 6.0.
#include "attention_launch.h"

namespace fp8k {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 512;                  // tokens per workgroup

__device__ __forceinline__ int32_t saturate(int64_t v) {
  return (int32_t)(v < 0x7fffffffll ? v : 0x7fffffffll);
}

// Lengths and their sums are below 2^32, so is what they are divided into.
__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, uint32_t page) {
  const uint32_t q = tokens / page;
  return q + (tokens - q * page != 0u ? 1u : 0u);
}

// kPer requests per thread and pass: one while the batch has at most 256
// (a shorter scan and search: 6.3 -> 4.9 us for 256 decoding requests), else 4.
template <int kPer>
__global__ __launch_bounds__(kThreads) void slot_map_kernel(SlotMapArgs a) {
  constexpr int kChunk = kThreads * kPer;     // requests per pass
  // of the pass's requests: first token and first block of each, relative to
  // the pass, and the tokens already cached
  __shared__ int64_t s_off[kChunk + 1];
  __shared__ int64_t s_first[kChunk];
  __shared__ int32_t s_have_tokens[kChunk];
  __shared__ int64_t s_wave[2][kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int64_t t1 = t0 + kTokens < a.T ? t0 + kTokens : a.T;
  const uint32_t page = (uint32_t)a.page;
  int64_t tok_base = 0, blk_base = 0;         // totals of the passes before
  for (int64_t r0 = 0; r0 < a.B; r0 += kChunk) {
    int64_t n[kPer], take[kPer], tn = 0, tb = 0;
    int32_t c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = r0 + tid * kPer + i;
      c[i] = 0;
      n[i] = 0;
      if (r < a.B) {
        const int32_t cc = a.computed[r], nn = a.fresh[r];
        c[i] = cc > 0 ? cc : 0;
        n[i] = nn > 0 ? nn : 0;
      }
      take[i] = blocks_of((uint32_t)c[i] + (uint32_t)n[i], page) - blocks_of((uint32_t)c[i], page);
      tn += n[i];
      tb += take[i];
    }
    int64_t xn = tn, xb = tb;                 // inclusive over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t un = __shfl_up(xn, d), ub = __shfl_up(xb, d);
      if (lane >= d) {
        xn += un;
        xb += ub;
      }
    }
    if (lane == 63) {
      s_wave[0][wave] = xn;
      s_wave[1][wave] = xb;
    }
    __syncthreads();
    int64_t on = xn - tn, ob = xb - tb, all_n = 0, all_b = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) {
        on += s_wave[0][w];
        ob += s_wave[1][w];
      }
      all_n += s_wave[0][w];
      all_b += s_wave[1][w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid * kPer + i;
      s_off[j] = on;
      s_first[j] = ob;
      s_have_tokens[j] = c[i];
      const int64_t r = r0 + j;
      if (blockIdx.x == 0 && r < a.B) {
        a.offsets[r] = saturate(tok_base + on);
        a.lens[r] = saturate((int64_t)c[i] + n[i]);
      }
      on += n[i];
      ob += take[i];
    }
    if (tid == 0) s_off[kChunk] = all_n;
    __syncthreads();

    // this workgroup's tokens among the pass's requests
    const int64_t lo = t0 > tok_base ? t0 : tok_base;
    const int64_t hi = t1 < tok_base + all_n ? t1 : tok_base + all_n;
    for (int64_t t = lo + tid; t < hi; t += kThreads) {
      const int64_t x = t - tok_base;
      int b = 0, e = kChunk;                  // last request whose first token is <= x
      while (e - b > 1) {
        const int m = (b + e) >> 1;
        if (s_off[m] <= x) b = m; else e = m;
      }
      const uint32_t cc = (uint32_t)s_have_tokens[b], pos = cc + (uint32_t)(x - s_off[b]);
      const uint32_t have = blocks_of(cc, page), i = pos / page;
      int64_t blk = -1;
      if (i < a.width) {
        if (i < have) {
          blk = a.table[(r0 + b) * a.ld_table + (int64_t)i];
        } else {
          const int64_t f = blk_base + s_first[b] + (i - have);
          if (f < a.num_free) blk = a.free_blocks[f];
        }
      }
      a.positions[t] = pos;
      a.slots[t] = blk < 0 ? -1 : blk * (int64_t)page + (pos - i * page);
    }

    // table entries of the pass's blocks, numbered as they are handed out; blocks
    // behind a row's end are passed over together, however many lengths ask for
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t f = (int64_t)blockIdx.x * kThreads + tid; f < all_b;) {
      int b = 0, e = kChunk;                  // last request whose first block is <= f
      while (e - b > 1) {
        const int m = (b + e) >> 1;
        if (s_first[m] <= f) b = m; else e = m;
      }
      const int64_t i = blocks_of((uint32_t)s_have_tokens[b], page) + (f - s_first[b]);
      if (i < a.width) {
        a.table[(r0 + b) * a.ld_table + i] =
            blk_base + f < a.num_free ? a.free_blocks[blk_base + f] : -1;
        f += stride;
      } else {
        const int64_t next = b + 1 < kChunk ? s_first[b + 1] : all_b;
        f += (next - f + stride - 1) / stride * stride;
      }
    }
    tok_base += all_n;
    blk_base += all_b;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.offsets[a.B] = saturate(tok_base);
    a.taken[0] = saturate(blk_base);
  }
  // behind the last token
  for (int64_t t = (t0 > tok_base ? t0 : tok_base) + tid; t < t1; t += kThreads) {
    a.positions[t] = -1;
    a.slots[t] = -1;
  }
}

}  // namespace

hipError_t launch_slot_map(const SlotMapArgs& a, hipStream_t st) {
  const int64_t grid = (a.T + kTokens - 1) / kTokens;
  const dim3 wgs((uint32_t)(grid > 0 ? grid : 1));
  if (a.B <= kThreads)
    hipLaunchKernelGGL(slot_map_kernel<1>, wgs, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL(slot_map_kernel<4>, wgs, dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace fp8k
