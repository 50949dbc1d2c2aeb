// Internal launchers behind the C ABI of fp8w8a8_step.h.  Arguments are already
// validated by the ABI layer (step_abi.hip); each launcher only enqueues kernels
// on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8k {

constexpr int64_t kMaxNormWidth = 65536;

struct NormQuantArgs {
  const uint16_t* x;
  const uint16_t* r;            // null: no residual
  uint16_t* r_out;
  const uint16_t* w;
  uint16_t* y;                  // null: not wanted
  uint8_t* q;                   // null: no quantization
  float* s;
  const float* scale;
  int64_t ld_x, ld_r, ld_ro, ld_y, ld_q, ld_s;
  int64_t T;
  int32_t H;
  float eps;
};
// mode: an FP8_SCALE_* value, looked at if a.q is set
hipError_t launch_norm_quant(const NormQuantArgs& a, int mode, hipStream_t st);

hipError_t launch_int4_pack(const uint8_t* values, int64_t ld_v, uint8_t* codes, int64_t N,
                            int64_t K, hipStream_t st);
hipError_t launch_int4_quant(const uint16_t* w, int64_t ld_w, uint8_t* codes, float* scales,
                             uint8_t* zeros, int64_t N, int64_t K, int group, hipStream_t st);

struct Int4Args {
  const uint16_t* x;
  int64_t ld_x;
  const uint8_t* codes;
  const float* scales;
  const uint8_t* zeros;         // null: 8 everywhere
  uint16_t* out;
  int64_t ld_out;
  int64_t M, N;
  int32_t K;
  float* parts;                 // [runs][M][N], or null: one run of K
};
// workspace bytes with which K is cut into runs (0: it is not)
size_t int4_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_int4_linear(const Int4Args& a, int group, hipStream_t st);
uint64_t int4_linear_items(int64_t M, int64_t N, int64_t K);

// (x - from) scale is ((x - from) pre) z.  The difference may be beyond fp32 where this is
// not, for scales below 1: pre is 0.5 for such, else 1.  scale log2(e) is c, in the kernels
// of far scales c pre post; it is beyond fp32 from 2.36e38 on: post is 2 there, else 1.
struct LogprobScale {
  float pre, z, c, post;
};
struct LogprobArgs {
  const void* logits;
  int64_t ld;
  const int64_t* tokens;
  float scale;
  int64_t T, V;
  int32_t k;
  float* logprobs;
  int32_t* ranks;
  float* entropy;
  float* lse;
  float* top;
  int32_t* ids;
  uint8_t* ws;
  LogprobScale unit;            // of `scale`, by the launcher
};
size_t logprobs_workspace(bool f32, int64_t T, int64_t V, int64_t k);
hipError_t launch_logprobs(LogprobArgs a, bool f32, hipStream_t st);
uint64_t logprobs_items(bool f32, int64_t T, int64_t V, int64_t k);

}  // namespace fp8k
