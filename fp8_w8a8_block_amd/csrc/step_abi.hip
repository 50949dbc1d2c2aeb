// C ABI of fp8w8a8_step.h: argument validation, device check and dispatch to the
// launchers.  Everything that the host can see is refused before anything is
// enqueued, in the order scheme, shape, NULL, stride, alignment, overlap, workspace.
#include <cmath>

#include "abi_common.h"
#include "attention_launch.h"
#include "fp8w8a8_attention.h"
#include "fp8w8a8_step.h"
#include "launch.h"
#include "step_launch.h"

namespace {

using namespace fp8abi;

// a contiguous vector of n elements (none behind a null pointer)
Range vec(const void* p, int64_t n, int64_t elem) { return range_of(p, 1, p ? n : 0, n, elem); }
Range mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  return range_of(p, p ? rows : 0, cols, ld, elem);
}

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

bool group_ok(int64_t group) { return group == 32 || group == 64 || group == 128; }

// shape of a weight [N, K] whose rows are cut into groups
bool weight_shape(int64_t N, int64_t K) {
  return N >= 0 && N < kMaxDim && K > 0 && K % 128 == 0 && K < kMaxDim && N <= kMaxElems / K;
}

// sizes of a product of M rows; a tile's rows of the weight are counted in 32 bits
bool product_shape(int64_t M, int64_t N, int64_t K) {
  return weight_shape(N, K) && N > 0 && K < ((int64_t)1 << 24) && M >= 0 && M < kMaxDim &&
         M <= kMaxElems / K && M <= kMaxElems / N;
}

// The axis of each of `half` pairs in the form that the kernel takes; false if the
// sections do not fit.
bool axes_of(int64_t A, const int64_t* sections, int order, int64_t half, fp8k::NormRopeArgs* a) {
  int64_t sum = 0;
  for (int64_t i = 0; i < A; ++i) {
    if (sections[i] < 0 || sections[i] > half) return false;
    sum += sections[i];
    if (order == FP8_AXES_IN_TURN && i > 0 && sections[i] > 0 &&
        i + A * (sections[i] - 1) >= half)
      return false;
  }
  if (sum != half) return false;
  int64_t axis = 0, end = sections[0];
  for (int64_t i = 0; i < half; ++i) {
    if (order == FP8_AXES_IN_TURN) {
      axis = i < A * sections[i % A] ? i % A : 0;
    } else {
      while (i >= end) end += sections[++axis];
    }
    a->axis_bits[i / 16] |= (uint32_t)axis << (i % 16 * 2);
  }
  a->axes = (int32_t)A;
  return true;
}

}  // namespace

extern "C" {

fp8_status fp8_validate_add_rms_norm_quant(const uint16_t* x, int64_t ld_x,
                                           const uint16_t* residual, int64_t ld_r,
                                           const uint16_t* residual_out, int64_t ld_ro,
                                           const uint16_t* weight, float eps, const uint16_t* y,
                                           int64_t ld_y, const uint8_t* q, int64_t ld_q,
                                           const float* scales, int64_t ld_s, int scale_mode,
                                           const float* scale, int64_t T, int64_t H) {
  const bool block = q && scale_mode == FP8_SCALE_BLOCK, row = q && scale_mode == FP8_SCALE_ROW;
  if (q && !block && !row && scale_mode != FP8_SCALE_TENSOR) return FP8_ERR_SCHEME;
  if (T < 0 || T >= kMaxDim || H <= 0 || H % 128 != 0 || H > fp8k::kMaxNormWidth)
    return FP8_ERR_SHAPE;
  // at most 1024 threads per row
  if ((uint64_t)T >= fp8k::kMaxGridItems / 1024u) return FP8_ERR_SHAPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return FP8_ERR_SHAPE;
  if (T == 0) return FP8_OK;
  if (!x || !weight || (!y && !q) || !residual != !residual_out) return FP8_ERR_NULL;
  if ((block || row) && !scales) return FP8_ERR_NULL;
  if (q && !block && !row && !scale) return FP8_ERR_NULL;
  const int64_t groups = block ? H / 128 : 1;
  if (ld_x < H || (residual && (ld_r < H || ld_ro < H)) || (y && ld_y < H) || (q && ld_q < H))
    return FP8_ERR_STRIDE;
  if ((block || row) && ld_s < groups) return FP8_ERR_STRIDE;
  if (!span_ok(T, ld_x) || (residual && (!span_ok(T, ld_r) || !span_ok(T, ld_ro))) ||
      (y && !span_ok(T, ld_y)) || (q && !span_ok(T, ld_q)) ||
      ((block || row) && !span_ok(T, ld_s)))
    return FP8_ERR_STRIDE;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
      !aligned(weight, 16) || !aligned(y, 16) || !aligned(q, 16) ||
      ((block || row) && !aligned(scales, 4)) || (q && !block && !row && !aligned(scale, 4)))
    return FP8_ERR_ALIGN;
  if (ld_x % 8 != 0 || (residual && (ld_r % 8 != 0 || ld_ro % 8 != 0)) || (y && ld_y % 8 != 0) ||
      (q && ld_q % 16 != 0))
    return FP8_ERR_ALIGN;
  const bool in_place = residual && residual == residual_out && ld_r == ld_ro;
  const Range outs[] = {mat(residual_out, T, H, ld_ro, 2), mat(y, T, H, ld_y, 2),
                        mat(q, T, H, ld_q, 1),
                        mat(block || row ? scales : nullptr, T, groups, ld_s, 4)};
  const Range ins[] = {mat(x, T, H, ld_x, 2), mat(in_place ? nullptr : residual, T, H, ld_r, 2),
                       vec(weight, H, 2), vec(q && !block && !row ? scale : nullptr, 1, 4)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_add_rms_norm_quant(const uint16_t* x, int64_t ld_x, const uint16_t* residual,
                                  int64_t ld_r, uint16_t* residual_out, int64_t ld_ro,
                                  const uint16_t* weight, float eps, uint16_t* y, int64_t ld_y,
                                  uint8_t* q, int64_t ld_q, float* scales, int64_t ld_s,
                                  int scale_mode, const float* scale, int64_t T, int64_t H,
                                  void* stream) {
  fp8_status st = fp8_validate_add_rms_norm_quant(x, ld_x, residual, ld_r, residual_out, ld_ro,
                                                  weight, eps, y, ld_y, q, ld_q, scales, ld_s,
                                                  scale_mode, scale, T, H);
  if (st != FP8_OK || T == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  fp8k::NormQuantArgs a = {};
  a.x = x;
  a.r = residual;
  a.r_out = residual_out;
  a.w = weight;
  a.y = y;
  a.q = q;
  a.s = scales;
  a.scale = scale;
  a.ld_x = ld_x;
  a.ld_r = ld_r;
  a.ld_ro = ld_ro;
  a.ld_y = ld_y;
  a.ld_q = ld_q;
  a.ld_s = ld_s;
  a.T = T;
  a.H = (int32_t)H;
  a.eps = eps;
  return launched(fp8k::launch_norm_quant(a, scale_mode, (hipStream_t)stream));
}

fp8_status fp8_validate_qk_norm_mrope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, int64_t ld_pos, int64_t A, const int64_t* sections, int axis_order,
    const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
    const uint16_t* query_out, int64_t ld_query_out, const uint8_t* key_cache,
    const uint8_t* value_cache, int64_t num_blocks, int64_t block_size, const float* k_scale,
    const float* v_scale) {
  if (axis_order != FP8_AXES_SECTIONS && axis_order != FP8_AXES_IN_TURN) return FP8_ERR_SCHEME;
  if (A < 1 || A > 4 || rot_dim < 0 || rot_dim > 512) return FP8_ERR_SHAPE;
  if (!sections) return FP8_ERR_NULL;
  fp8k::NormRopeArgs a = {};
  if (!axes_of(A, sections, axis_order, rot_dim / 2, &a)) return FP8_ERR_SHAPE;
  const fp8_status st = fp8_validate_qk_norm_rope_cache(
      query, ld_query, key, ld_key, value, ld_value, q_weight, k_weight, eps, cos_sin, max_pos,
      rot_dim, interleaved, positions, slot_mapping, T, Hq, Hk, D, query_out, ld_query_out,
      key_cache, value_cache, num_blocks, block_size, k_scale, v_scale);
  if (st != FP8_OK || T == 0) return st;
  // the axes behind the first
  if (A > 1 && (ld_pos < T || !span_ok(A, ld_pos))) return FP8_ERR_STRIDE;
  const int64_t cap = num_blocks * block_size;
  const Range all = mat(positions, A, T, ld_pos, 8);
  const Range outs[] = {mat(query_out, T, Hq * D, ld_query_out, 2),
                        mat(key_cache, cap, Hk * D, Hk * D, 1),
                        mat(value_cache, cap, Hk * D, Hk * D, 1)};
  for (const Range& o : outs)
    if (overlap(o, all)) return FP8_ERR_ALIAS;
  return FP8_OK;
}

fp8_status fp8_qk_norm_mrope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, int64_t ld_pos, int64_t A, const int64_t* sections, int axis_order,
    const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk, int64_t D, uint16_t* query_out,
    int64_t ld_query_out, uint8_t* key_cache, uint8_t* value_cache, int64_t num_blocks,
    int64_t block_size, const float* k_scale, const float* v_scale, void* stream) {
  fp8_status st = fp8_validate_qk_norm_mrope_cache(
      query, ld_query, key, ld_key, value, ld_value, q_weight, k_weight, eps, cos_sin, max_pos,
      rot_dim, interleaved, positions, ld_pos, A, sections, axis_order, slot_mapping, T, Hq, Hk, D,
      query_out, ld_query_out, key_cache, value_cache, num_blocks, block_size, k_scale, v_scale);
  if (st != FP8_OK || T == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  fp8k::NormRopeArgs a = {};
  axes_of(A, sections, axis_order, rot_dim / 2, &a);
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
  a.ld_pos = ld_pos;
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

fp8_status fp8_validate_int4_pack(const uint8_t* values, int64_t ld_v, const uint8_t* codes,
                                  int64_t N, int64_t K) {
  if (!weight_shape(N, K)) return FP8_ERR_SHAPE;
  if (N == 0) return FP8_OK;
  if (!values || !codes) return FP8_ERR_NULL;
  if (ld_v < K || !span_ok(N, ld_v)) return FP8_ERR_STRIDE;
  if (!aligned(values, 8) || ld_v % 8 != 0 || !aligned(codes, 16)) return FP8_ERR_ALIGN;
  return overlap(mat(values, N, K, ld_v, 1), vec(codes, N * (K / 2), 1)) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_int4_pack(const uint8_t* values, int64_t ld_v, uint8_t* codes, int64_t N, int64_t K,
                         void* stream) {
  fp8_status st = fp8_validate_int4_pack(values, ld_v, codes, N, K);
  if (st != FP8_OK || N == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  return launched(fp8k::launch_int4_pack(values, ld_v, codes, N, K, (hipStream_t)stream));
}

fp8_status fp8_validate_int4_quant_weight(const uint16_t* w, int64_t ld_w, const uint8_t* codes,
                                          const float* scales, const uint8_t* zeros, int64_t N,
                                          int64_t K, int64_t group) {
  if (!group_ok(group)) return FP8_ERR_BLOCK;
  if (!weight_shape(N, K)) return FP8_ERR_SHAPE;
  if (N == 0) return FP8_OK;
  if (!w || !codes || !scales) return FP8_ERR_NULL;
  if (ld_w < K || !span_ok(N, ld_w)) return FP8_ERR_STRIDE;
  if (!aligned(w, 16) || ld_w % 8 != 0 || !aligned(codes, 16) || !aligned(scales, 4))
    return FP8_ERR_ALIGN;
  const Range outs[] = {vec(codes, N * (K / 2), 1), vec(scales, N * (K / group), 4),
                        vec(zeros, N * (K / group), 1)};
  const Range ins[] = {mat(w, N, K, ld_w, 2)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_int4_quant_weight(const uint16_t* w, int64_t ld_w, uint8_t* codes, float* scales,
                                 uint8_t* zeros, int64_t N, int64_t K, int64_t group,
                                 void* stream) {
  fp8_status st = fp8_validate_int4_quant_weight(w, ld_w, codes, scales, zeros, N, K, group);
  if (st != FP8_OK || N == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  return launched(fp8k::launch_int4_quant(w, ld_w, codes, scales, zeros, N, K, (int)group,
                                          (hipStream_t)stream));
}

fp8_status fp8_validate_int4_linear(const uint16_t* x, int64_t ld_x, const uint8_t* codes,
                                    const float* scales, const uint8_t* zeros, int64_t group,
                                    const uint16_t* out, int64_t ld_out, int64_t M, int64_t N,
                                    int64_t K, const void* workspace, size_t ws_bytes) {
  if (!group_ok(group)) return FP8_ERR_BLOCK;
  if (!product_shape(M, N, K)) return FP8_ERR_SHAPE;
  if (M > 0 && fp8k::int4_linear_items(M, N, K) >= fp8k::kMaxGridItems) return FP8_ERR_SHAPE;
  if (M == 0) return FP8_OK;
  if (!x || !codes || !scales || !out) return FP8_ERR_NULL;
  if (ld_x < K || ld_out < N || !span_ok(M, ld_x) || !span_ok(M, ld_out)) return FP8_ERR_STRIDE;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 2) ||
      ld_x % 8 != 0)
    return FP8_ERR_ALIGN;
  const Range o = mat(out, M, N, ld_out, 2);
  const Range ins[] = {mat(x, M, K, ld_x, 2), vec(codes, N * (K / 2), 1),
                       vec(scales, N * (K / group), 4), vec(zeros, N * (K / group), 1)};
  for (const Range& r : ins)
    if (overlap(o, r)) return FP8_ERR_ALIAS;
  if (!workspace) return FP8_OK;
  if (!aligned(workspace, 16)) return FP8_ERR_WORKSPACE;
  const Range ws = {(uintptr_t)workspace, (uintptr_t)workspace + ws_bytes};
  for (const Range& r : ins)
    if (overlap(ws, r)) return FP8_ERR_ALIAS;
  return overlap(ws, o) ? FP8_ERR_ALIAS : FP8_OK;
}

size_t fp8_int4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || !product_shape(M, N, K)) return 0;
  return fp8k::int4_workspace(M, N, K);
}

fp8_status fp8_int4_linear(const uint16_t* x, int64_t ld_x, const uint8_t* codes,
                           const float* scales, const uint8_t* zeros, int64_t group, uint16_t* out,
                           int64_t ld_out, int64_t M, int64_t N, int64_t K, void* workspace,
                           size_t ws_bytes, void* stream) {
  fp8_status st = fp8_validate_int4_linear(x, ld_x, codes, scales, zeros, group, out, ld_out, M, N,
                                           K, workspace, ws_bytes);
  if (st != FP8_OK || M == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  fp8k::Int4Args a = {};
  a.x = x;
  a.ld_x = ld_x;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.out = out;
  a.ld_out = ld_out;
  a.M = M;
  a.N = N;
  a.K = (int32_t)K;
  const size_t need = fp8k::int4_workspace(M, N, K);
  a.parts = workspace && need > 0 && ws_bytes >= need ? (float*)workspace : nullptr;
  return launched(fp8k::launch_int4_linear(a, (int)group, (hipStream_t)stream));
}

}  // extern "C"

namespace {

bool logits_shape(int type, int64_t T, int64_t V, int64_t k) {
  if (type != FP8_LOGITS_BF16 && type != FP8_LOGITS_F32) return false;
  return T >= 0 && T < kMaxDim && V >= 1 && V < kMaxDim && T <= kMaxElems / V && k >= 0 &&
         k <= FP8_MAX_TOP && k <= V &&
         (T == 0 || fp8k::logprobs_items(type == FP8_LOGITS_F32, T, V, k) < fp8k::kMaxGridItems);
}

}  // namespace

extern "C" {

size_t fp8_logprobs_workspace_bytes(int logits_type, int64_t T, int64_t V, int64_t k) {
  if (!logits_shape(logits_type, T, V, k) || T == 0) return 0;
  return fp8k::logprobs_workspace(logits_type == FP8_LOGITS_F32, T, V, k);
}

fp8_status fp8_validate_token_logprobs(const void* logits, int logits_type, int64_t ld,
                                       const int64_t* tokens, float scale, int64_t T, int64_t V,
                                       int64_t k, const float* logprobs, const int32_t* ranks,
                                       const float* entropy, const float* lse,
                                       const float* top_logprobs, const int32_t* top_ids,
                                       const void* workspace, size_t ws_bytes, size_t ws_needed) {
  if (logits_type != FP8_LOGITS_BF16 && logits_type != FP8_LOGITS_F32) return FP8_ERR_SCHEME;
  if (!logits_shape(logits_type, T, V, k) || !(scale > 0.0f) || std::isinf(scale))
    return FP8_ERR_SHAPE;
  if (T == 0) return FP8_OK;
  if (!logits || !tokens || !logprobs || !ranks || !entropy || !lse) return FP8_ERR_NULL;
  if (k > 0 && (!top_logprobs || !top_ids)) return FP8_ERR_NULL;
  if (ld < V || !span_ok(T, ld)) return FP8_ERR_STRIDE;
  const int64_t size = logits_type == FP8_LOGITS_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(tokens, 8) || !aligned(logprobs, 4) ||
      !aligned(ranks, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
      (k > 0 && (!aligned(top_logprobs, 4) || !aligned(top_ids, 4))))
    return FP8_ERR_ALIGN;
  if (ws_needed > 0 && (!workspace || ws_bytes < ws_needed || !aligned(workspace, 16)))
    return FP8_ERR_WORKSPACE;
  const Range outs[] = {vec(logprobs, T, 4), vec(ranks, T, 4), vec(entropy, T, 4), vec(lse, T, 4),
                        vec(k > 0 ? top_logprobs : nullptr, T * k, 4),
                        vec(k > 0 ? top_ids : nullptr, T * k, 4),
                        {(uintptr_t)workspace, (uintptr_t)workspace + ws_needed}};
  const Range ins[] = {mat(logits, T, V, ld, size), vec(tokens, T, 8)};
  return any_overlap(outs, ins) ? FP8_ERR_ALIAS : FP8_OK;
}

fp8_status fp8_token_logprobs(const void* logits, int logits_type, int64_t ld,
                              const int64_t* tokens, float scale, int64_t T, int64_t V, int64_t k,
                              float* logprobs, int32_t* ranks, float* entropy, float* lse,
                              float* top_logprobs, int32_t* top_ids, void* workspace,
                              size_t ws_bytes, void* stream) {
  fp8_status st = fp8_validate_token_logprobs(
      logits, logits_type, ld, tokens, scale, T, V, k, logprobs, ranks, entropy, lse, top_logprobs,
      top_ids, workspace, ws_bytes, fp8_logprobs_workspace_bytes(logits_type, T, V, k));
  if (st != FP8_OK || T == 0) return st;
  if ((st = check_device()) != FP8_OK) return st;
  fp8k::LogprobArgs a = {};
  a.logits = logits;
  a.ld = T > 1 ? ld : V;
  a.tokens = tokens;
  a.scale = scale;
  a.T = T;
  a.V = V;
  a.k = (int32_t)k;
  a.logprobs = logprobs;
  a.ranks = ranks;
  a.entropy = entropy;
  a.lse = lse;
  a.top = top_logprobs;
  a.ids = top_ids;
  a.ws = (uint8_t*)workspace;
  return launched(fp8k::launch_logprobs(a, logits_type == FP8_LOGITS_F32, (hipStream_t)stream));
}

}  // extern "C"
