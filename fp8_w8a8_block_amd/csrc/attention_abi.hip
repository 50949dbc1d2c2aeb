// C ABI of the paged attention step: argument validation, device check and
// dispatch to the launchers.  The checks follow those of the KV-cache calls in
// abi.hip: everything that the host can see is refused before anything is
// enqueued, in the order shape, NULL, stride, alignment, overlap, workspace.
#include <cmath>

#include "abi_common.h"
#include "attention_launch.h"
#include "fp8w8a8_attention.h"
#include "launch.h"

namespace {

using namespace fp8abi;

// shape of a paged cache with H heads of D
fp8_status cache_shape(int64_t num_blocks, int64_t block_size, int64_t H, int64_t D) {
  if (H <= 0 || D <= 0 || H >= kMaxDim || D >= kMaxDim || H * D >= kMaxDim) return FP8_ERR_SHAPE;
  if (num_blocks < 0 || num_blocks >= kMaxDim || block_size <= 0 || block_size >= kMaxDim)
    return FP8_ERR_SHAPE;
  if (num_blocks * block_size > kMaxElems / (H * D)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

// a contiguous vector of n elements
Range vec(const void* p, int64_t n, int64_t elem) { return range_of(p, 1, n, n, elem); }

template <int N, int M>
bool any_overlap(const Range (&outs)[N], const Range (&ins)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

fp8_status fp8_validate_kv_slot_map(const int32_t* computed_lens, const int32_t* new_lens,
                                    int64_t B, int64_t block_size, const int32_t* block_table,
                                    int64_t ld_table, int64_t table_width,
                                    const int32_t* free_blocks, int64_t num_free,
                                    const int64_t* slot_mapping, const int64_t* positions,
                                    int64_t T, const int32_t* query_offsets,
                                    const int32_t* seq_lens, const int32_t* blocks_taken) {
  if (B < 0 || B >= kMaxDim || T < 0 || T >= kMaxDim || block_size <= 0 || block_size >= kMaxDim ||
      table_width < 0 || table_width >= kMaxDim || num_free < 0 || num_free >= kMaxDim)
    return FP8_ERR_SHAPE;
  if (!query_offsets || !blocks_taken) return FP8_ERR_NULL;
  if (B > 0 && (!computed_lens || !new_lens || !seq_lens)) return FP8_ERR_NULL;
  if (B > 0 && table_width > 0 && !block_table) return FP8_ERR_NULL;
  if (num_free > 0 && !free_blocks) return FP8_ERR_NULL;
  if (T > 0 && (!slot_mapping || !positions)) return FP8_ERR_NULL;
  if (B > 0 && (ld_table < table_width || !span_ok(B, ld_table))) return FP8_ERR_STRIDE;
  if (!aligned(computed_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_blocks, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 8) ||
      !aligned(query_offsets, 4) || !aligned(seq_lens, 4) || !aligned(blocks_taken, 4))
    return FP8_ERR_ALIGN;
  const Range outs[] = {range_of(block_table, B, table_width, ld_table, 4),
                        vec(slot_mapping, T, 8),
                        vec(positions, T, 8),
                        vec(query_offsets, B + 1, 4),
                        vec(seq_lens, B, 4),
                        vec(blocks_taken, 1, 4)};
  const Range ins[] = {vec(computed_lens, B, 4), vec(new_lens, B, 4), vec(free_blocks, num_free, 4)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_kv_slot_map(const int32_t* computed_lens, const int32_t* new_lens, int64_t B,
                           int64_t block_size, int32_t* block_table, int64_t ld_table,
                           int64_t table_width, const int32_t* free_blocks, int64_t num_free,
                           int64_t* slot_mapping, int64_t* positions, int64_t T,
                           int32_t* query_offsets, int32_t* seq_lens, int32_t* blocks_taken,
                           void* stream) {
  fp8_status st = fp8_validate_kv_slot_map(computed_lens, new_lens, B, block_size, block_table,
                                           ld_table, table_width, free_blocks, num_free,
                                           slot_mapping, positions, T, query_offsets, seq_lens,
                                           blocks_taken);
  if (st != FP8_OK) return st;
  if ((st = check_device()) != FP8_OK) return st;
  const fp8k::SlotMapArgs a = {computed_lens, new_lens,     B,         (int32_t)block_size,
                               block_table,   ld_table,     table_width, free_blocks,
                               num_free,      slot_mapping, positions, T,
                               query_offsets, seq_lens,     blocks_taken};
  return launched(fp8k::launch_slot_map(a, (hipStream_t)stream));
}

fp8_status fp8_validate_qk_norm_rope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk,
    int64_t D, const uint16_t* query_out, int64_t ld_query_out, const uint8_t* key_cache,
    const uint8_t* value_cache, int64_t num_blocks, int64_t block_size, const float* k_scale,
    const float* v_scale) {
  (void)interleaved;
  const fp8_status st = cache_shape(num_blocks, block_size, Hk, D);
  if (st != FP8_OK) return st;
  if (T < 0 || T >= kMaxDim || Hq <= 0 || Hq >= kMaxDim || D % 16 != 0 || D > 512)
    return FP8_ERR_SHAPE;
  if (Hq + 2 * Hk >= kMaxDim || T > kMaxElems / ((Hq + 2 * Hk) * D)) return FP8_ERR_SHAPE;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0 || max_pos < 0 || max_pos >= kMaxDim)
    return FP8_ERR_SHAPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return FP8_ERR_SHAPE;
  if (T > 0 && fp8k::norm_rope_items(T, Hq, Hk, D) >= fp8k::kMaxGridItems) return FP8_ERR_SHAPE;
  if (T == 0) return FP8_OK;
  const int64_t cap = num_blocks * block_size, hq = Hq * D, hk = Hk * D;
  if (!query || !key || !value || !q_weight || !k_weight || !positions || !slot_mapping ||
      !query_out || !k_scale || !v_scale)
    return FP8_ERR_NULL;
  if (rot_dim > 0 && max_pos > 0 && !cos_sin) return FP8_ERR_NULL;
  if (cap > 0 && (!key_cache || !value_cache)) return FP8_ERR_NULL;
  if (ld_query < hq || ld_key < hk || ld_value < hk || ld_query_out < hq) return FP8_ERR_STRIDE;
  if (!span_ok(T, ld_query) || !span_ok(T, ld_key) || !span_ok(T, ld_value) ||
      !span_ok(T, ld_query_out))
    return FP8_ERR_STRIDE;
  if (!aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(cos_sin, 16) || !aligned(query_out, 16) ||
      !aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(positions, 8) ||
      !aligned(slot_mapping, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return FP8_ERR_ALIGN;
  if (ld_query % 8 != 0 || ld_key % 8 != 0 || ld_value % 8 != 0 || ld_query_out % 8 != 0)
    return FP8_ERR_ALIGN;
  const Range outs[] = {range_of(query_out, T, hq, ld_query_out, 2),
                        range_of(key_cache, cap, hk, hk, 1), range_of(value_cache, cap, hk, hk, 1)};
  const Range ins[] = {range_of(query, T, hq, ld_query, 2),
                       range_of(key, T, hk, ld_key, 2),
                       range_of(value, T, hk, ld_value, 2),
                       vec(q_weight, D, 2),
                       vec(k_weight, D, 2),
                       range_of(cos_sin, max_pos, rot_dim, rot_dim, 4),
                       vec(positions, T, 8),
                       vec(slot_mapping, T, 8),
                       vec(k_scale, 1, 4),
                       vec(v_scale, 1, 4)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_qk_norm_rope_cache(const uint16_t* query, int64_t ld_query, const uint16_t* key,
                                  int64_t ld_key, const uint16_t* value, int64_t ld_value,
                                  const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                  const float* cos_sin, int64_t max_pos, int64_t rot_dim,
                                  int interleaved, const int64_t* positions,
                                  const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk,
                                  int64_t D, uint16_t* query_out, int64_t ld_query_out,
                                  uint8_t* key_cache, uint8_t* value_cache, int64_t num_blocks,
                                  int64_t block_size, const float* k_scale, const float* v_scale,
                                  void* stream) {
  fp8_status st = fp8_validate_qk_norm_rope_cache(
      query, ld_query, key, ld_key, value, ld_value, q_weight, k_weight, eps, cos_sin, max_pos,
      rot_dim, interleaved, positions, slot_mapping, T, Hq, Hk, D, query_out, ld_query_out,
      key_cache, value_cache, num_blocks, block_size, k_scale, v_scale);
  if (st != FP8_OK || T == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  fp8k::NormRopeArgs a = {};
  a.q = query;
  a.k = key;
  a.v = value;
  a.ld_q = ld_query;
  a.ld_k = ld_key;
  a.ld_v = ld_value;
  a.qw = q_weight;
  a.kw = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_pos = max_pos;
  a.rot = (int32_t)rot_dim;
  a.positions = positions;
  a.slots = slot_mapping;
  a.T = T;
  a.Hq = (int32_t)Hq;
  a.Hk = (int32_t)Hk;
  a.D = (int32_t)D;
  a.q_out = query_out;
  a.ld_qo = ld_query_out;
  a.kc = key_cache;
  a.vc = value_cache;
  a.capacity = num_blocks * block_size;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return launched(fp8k::launch_norm_rope(a, interleaved != 0, (hipStream_t)stream));
}

}  // extern "C"

namespace {

// sizes that the kernels are built for
bool attention_sizes(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D) {
  if (T < 0 || T >= kMaxDim || B < 0 || B >= kMaxDim || Hk <= 0 || Hq <= 0 || Hq >= kMaxDim ||
      Hq % Hk != 0)
    return false;
  if (D != 64 && D != 128 && D != 256) return false;
  // rows of a KV head, and (tokens, head) pairs, are counted in 32 bits
  return Hq * D < kMaxDim && T < kMaxDim / Hq;
}

}  // namespace

extern "C" {

size_t fp8_attention_workspace_bytes(int shared_prefix, int64_t T, int64_t B, int64_t Hq,
                                     int64_t Hk, int64_t D) {
  if (!attention_sizes(T, B, Hq, Hk, D) || T == 0 || B == 0) return 0;
  return fp8k::attention_workspace(shared_prefix != 0, T, B, Hq, Hk, D);
}

fp8_status fp8_validate_attention(const uint16_t* query, int64_t ld_query,
                                  const uint8_t* key_cache, const uint8_t* value_cache,
                                  int64_t num_blocks, int64_t block_size,
                                  const int32_t* prefix_table, int64_t prefix_width,
                                  const int32_t* prefix_len, const int32_t* block_table,
                                  int64_t ld_table, int64_t table_width, const int32_t* seq_lens,
                                  const int32_t* query_offsets, int64_t B, const float* k_scale,
                                  const float* v_scale, float scale, int64_t window, int64_t sinks,
                                  const uint16_t* out, int64_t ld_out, const float* lse, int64_t T,
                                  int64_t Hq, int64_t Hk, int64_t D, const void* workspace,
                                  size_t ws_bytes, size_t ws_needed) {
  const bool prefix = prefix_table || prefix_len || prefix_width != 0;
  const fp8_status st = cache_shape(num_blocks, block_size, Hk, D);
  if (st != FP8_OK) return st;
  if (!attention_sizes(T, B, Hq, Hk, D) || num_blocks * block_size >= kMaxDim)
    return FP8_ERR_SHAPE;
  if (table_width < 0 || table_width >= kMaxDim || prefix_width < 0 || prefix_width >= kMaxDim ||
      window < 0 || window >= kMaxDim || sinks < 0 || sinks >= kMaxDim || !std::isfinite(scale))
    return FP8_ERR_SHAPE;
  if (T == 0 || B == 0) return FP8_OK;
  const int64_t cap = num_blocks * block_size, hq = Hq * D, hk = Hk * D;
  if (!query || !seq_lens || !query_offsets || !k_scale || !v_scale || !out) return FP8_ERR_NULL;
  if (cap > 0 && (!key_cache || !value_cache)) return FP8_ERR_NULL;
  if (table_width > 0 && !block_table) return FP8_ERR_NULL;
  if (prefix && (!prefix_len || (prefix_width > 0 && !prefix_table))) return FP8_ERR_NULL;
  if (ld_query < hq || ld_out < hq || ld_table < table_width) return FP8_ERR_STRIDE;
  if (!span_ok(T, ld_query) || !span_ok(T, ld_out) || !span_ok(B, ld_table)) return FP8_ERR_STRIDE;
  if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
      !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(query_offsets, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(prefix_table, 4) || !aligned(prefix_len, 4))
    return FP8_ERR_ALIGN;
  if (ld_query % 8 != 0 || ld_out % 8 != 0) return FP8_ERR_ALIGN;
  if (ws_needed > 0 && (!workspace || ws_bytes < ws_needed || !aligned(workspace, 16)))
    return FP8_ERR_WORKSPACE;
  const Range outs[] = {range_of(out, T, hq, ld_out, 2), vec(lse, lse ? T * Hq : 0, 4),
                        {(uintptr_t)workspace, (uintptr_t)workspace + ws_needed}};
  const Range ins[] = {range_of(query, T, hq, ld_query, 2),
                       range_of(key_cache, cap, hk, hk, 1),
                       range_of(value_cache, cap, hk, hk, 1),
                       range_of(block_table, B, table_width, ld_table, 4),
                       vec(prefix_table, prefix_width, 4),
                       vec(prefix_len, prefix_len ? 1 : 0, 4),
                       vec(seq_lens, B, 4),
                       vec(query_offsets, B + 1, 4),
                       vec(k_scale, 1, 4),
                       vec(v_scale, 1, 4)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

}  // extern "C"

namespace {

fp8_status attention(const uint16_t* query, int64_t ld_query, const uint8_t* key_cache,
                     const uint8_t* value_cache, int64_t num_blocks, int64_t block_size,
                     const int32_t* prefix_table, int64_t prefix_width, const int32_t* prefix_len,
                     const int32_t* block_table, int64_t ld_table, int64_t table_width,
                     const int32_t* seq_lens, const int32_t* query_offsets, int64_t B,
                     const float* k_scale, const float* v_scale, float scale, int64_t window,
                     int64_t sinks, uint16_t* out, int64_t ld_out, float* lse, int64_t T,
                     int64_t Hq, int64_t Hk, int64_t D, void* workspace, size_t ws_bytes,
                     void* stream) {
  // the workspace's size depends on the device, so everything else comes first
  fp8_status st = fp8_validate_attention(
      query, ld_query, key_cache, value_cache, num_blocks, block_size, prefix_table, prefix_width,
      prefix_len, block_table, ld_table, table_width, seq_lens, query_offsets, B, k_scale, v_scale,
      scale, window, sinks, out, ld_out, lse, T, Hq, Hk, D, workspace, ws_bytes, 0);
  if (st != FP8_OK || T == 0 || B == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  const size_t need = fp8_attention_workspace_bytes(prefix_len != nullptr, T, B, Hq, Hk, D);
  st = fp8_validate_attention(query, ld_query, key_cache, value_cache, num_blocks, block_size,
                              prefix_table, prefix_width, prefix_len, block_table, ld_table,
                              table_width, seq_lens, query_offsets, B, k_scale, v_scale, scale,
                              window, sinks, out, ld_out, lse, T, Hq, Hk, D, workspace, ws_bytes,
                              need);
  if (st != FP8_OK) return st;
  fp8k::AttentionArgs a = {};
  a.q = query;
  a.ld_q = ld_query;
  a.kc = key_cache;
  a.vc = value_cache;
  a.num_blocks = (int32_t)num_blocks;
  a.page = (int32_t)block_size;
  a.table = block_table;
  a.ld_table = ld_table;
  a.width = (int32_t)table_width;
  a.lens = seq_lens;
  a.offsets = query_offsets;
  a.B = (int32_t)B;
  a.prefix_table = prefix_table;
  a.prefix_width = (int32_t)prefix_width;
  a.prefix_len = prefix_len;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.scale = scale;
  a.window = (int32_t)window;
  a.sinks = (int32_t)sinks;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.T = (int32_t)T;
  a.Hq = (int32_t)Hq;
  a.Hk = (int32_t)Hk;
  a.G = (int32_t)(Hq / Hk);
  a.inv_G = 1.0 / (double)a.G;
  a.inv_page = 1.0 / (double)a.page;
  a.ws = (uint8_t*)workspace;
  return launched(fp8k::launch_attention(a, (int)D, (hipStream_t)stream));
}

}  // namespace

extern "C" {

fp8_status fp8_paged_attention(const uint16_t* query, int64_t ld_query, const uint8_t* key_cache,
                               const uint8_t* value_cache, int64_t num_blocks, int64_t block_size,
                               const int32_t* block_table, int64_t ld_table, int64_t table_width,
                               const int32_t* seq_lens, const int32_t* query_offsets, int64_t B,
                               const float* k_scale, const float* v_scale, float scale,
                               int64_t window, int64_t sinks, uint16_t* out, int64_t ld_out,
                               float* lse, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                               void* workspace, size_t ws_bytes, void* stream) {
  return attention(query, ld_query, key_cache, value_cache, num_blocks, block_size, nullptr, 0,
                   nullptr, block_table, ld_table, table_width, seq_lens, query_offsets, B, k_scale,
                   v_scale, scale, window, sinks, out, ld_out, lse, T, Hq, Hk, D, workspace,
                   ws_bytes, stream);
}

fp8_status fp8_prefix_attention(const uint16_t* query, int64_t ld_query, const uint8_t* key_cache,
                                const uint8_t* value_cache, int64_t num_blocks, int64_t block_size,
                                const int32_t* prefix_table, int64_t prefix_width,
                                const int32_t* prefix_len, const int32_t* block_table,
                                int64_t ld_table, int64_t table_width, const int32_t* seq_lens,
                                const int32_t* query_offsets, int64_t B, const float* k_scale,
                                const float* v_scale, float scale, uint16_t* out, int64_t ld_out,
                                float* lse, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                void* workspace, size_t ws_bytes, void* stream) {
  if (T > 0 && B > 0 && !prefix_len) return FP8_ERR_NULL;
  return attention(query, ld_query, key_cache, value_cache, num_blocks, block_size, prefix_table,
                   prefix_width, prefix_len, block_table, ld_table, table_width, seq_lens,
                   query_offsets, B, k_scale, v_scale, scale, 0, 0, out, ld_out, lse, T, Hq, Hk, D,
                   workspace, ws_bytes, stream);
}

}  // extern "C"
