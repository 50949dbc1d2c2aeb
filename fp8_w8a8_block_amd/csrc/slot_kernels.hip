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
// time (4 per thread, a wave scan, a scan over the waves), and answers for its
// own stretch of tokens and its own requests' table entries.  A token of a
// block that this step hands out reads the free list, not the table entry that
// another workgroup may be writing, so no workgroup waits for another.  The
// sums cost a few microseconds of latency per 1024 requests, less than a
// second launch that would read them.
#include "attention_launch.h"

namespace fp8k {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                       // requests per thread
constexpr int kChunk = kThreads * kPer;       // requests per pass
constexpr int kTokens = 512;                  // tokens per workgroup

__device__ __forceinline__ int32_t saturate(int64_t v) {
  return (int32_t)(v < 0x7fffffffll ? v : 0x7fffffffll);
}

__global__ __launch_bounds__(kThreads) void slot_map_kernel(SlotMapArgs a) {
  // of the pass's requests: first token and first block of each, relative to
  // the pass, and the tokens already cached
  __shared__ int64_t s_off[kChunk + 1];
  __shared__ int64_t s_first[kChunk];
  __shared__ int32_t s_have_tokens[kChunk];
  __shared__ int64_t s_wave[2][kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int64_t t1 = t0 + kTokens < a.T ? t0 + kTokens : a.T;
  const int64_t page = a.page;
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
      const int64_t have = ((int64_t)c[i] + page - 1) / page;
      take[i] = ((int64_t)c[i] + n[i] + page - 1) / page - have;
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
      const int64_t cc = s_have_tokens[b], pos = cc + (x - s_off[b]);
      const int64_t have = (cc + page - 1) / page, i = pos / page;
      int64_t blk = -1;
      if (i < a.width) {
        if (i < have) {
          blk = a.table[(r0 + b) * a.ld_table + i];
        } else {
          const int64_t f = blk_base + s_first[b] + (i - have);
          if (f < a.num_free) blk = a.free_blocks[f];
        }
      }
      a.positions[t] = pos;
      a.slots[t] = blk < 0 ? -1 : blk * page + (pos - i * page);
    }

    // table entries of requests r0 + wg, r0 + wg + grid, ...
    for (int64_t j = blockIdx.x; j < kChunk && r0 + j < a.B; j += gridDim.x) {
      const int64_t cc = s_have_tokens[j], nn = s_off[j + 1] - s_off[j];
      const int64_t have = (cc + page - 1) / page;
      int64_t need = (cc + nn + page - 1) / page;
      need = need < a.width ? need : a.width;
      for (int64_t i = have + tid; i < need; i += kThreads) {
        const int64_t f = blk_base + s_first[j] + (i - have);
        a.table[(r0 + j) * a.ld_table + i] = f < a.num_free ? a.free_blocks[f] : -1;
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
  hipLaunchKernelGGL(slot_map_kernel, dim3((uint32_t)(grid > 0 ? grid : 1)), dim3(kThreads), 0, st,
                     a);
  return hipGetLastError();
}

}  // namespace fp8k
