// Internal launchers behind the C ABI of the paged attention step.
// Arguments are already validated by the ABI layer (attention_abi.hip); each
// launcher only enqueues kernels on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8k {

struct SlotMapArgs {
  const int32_t* computed;
  const int32_t* fresh;
  int64_t B;
  int32_t page;                 // tokens per block
  int32_t* table;
  int64_t ld_table, width;
  const int32_t* free_blocks;
  int64_t num_free;
  int64_t* slots;
  int64_t* positions;
  int64_t T;
  int32_t* offsets;
  int32_t* lens;
  int32_t* taken;
};
hipError_t launch_slot_map(const SlotMapArgs& a, hipStream_t st);

struct NormRopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ld_q, ld_k, ld_v;
  const uint16_t* qw;
  const uint16_t* kw;
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int32_t rot;
  const int64_t* positions;
  const int64_t* slots;
  int64_t T;
  int32_t Hq, Hk, D;
  uint16_t* q_out;
  int64_t ld_qo;
  uint8_t* kc;
  uint8_t* vc;
  int64_t capacity;             // slots of the cache
  const float* k_scale;
  const float* v_scale;
};
hipError_t launch_norm_rope(const NormRopeArgs& a, bool interleaved, hipStream_t st);

struct AttentionArgs {
  const uint16_t* q;
  int64_t ld_q;
  const uint8_t* kc;
  const uint8_t* vc;
  int32_t num_blocks, page;     // page: tokens per block
  const int32_t* table;
  int64_t ld_table;
  int32_t width;
  const int32_t* lens;
  const int32_t* offsets;
  int32_t B;
  const int32_t* prefix_table;
  int32_t prefix_width;
  const int32_t* prefix_len;    // null: no shared prefix
  const float* k_scale;
  const float* v_scale;
  float scale;
  int32_t window, sinks;
  uint16_t* out;
  int64_t ld_out;
  float* lse;
  int32_t T, Hq, Hk, G;         // G = Hq / Hk
  double inv_G, inv_page;       // 1 / G, 1 / page
  uint8_t* ws;
};
// Workspace bytes of launch_attention for these sizes on the current device.
size_t attention_workspace(bool prefix, int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D);
hipError_t launch_attention(const AttentionArgs& a, int D, hipStream_t st);

// work-items of the largest grid of these calls (see kMaxGridItems)
uint64_t norm_rope_items(int64_t T, int64_t Hq, int64_t Hk, int64_t D);

}  // namespace fp8k
