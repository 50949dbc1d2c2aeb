/*
 * fp8w8a8_step.h -- C ABI of what a serving step runs around the FP8 linears
 * of fp8w8a8.h and the paged attention of fp8w8a8_attention.h, for gfx950:
 *   1. fp8_add_rms_norm_quant: the residual's addition, the RMS norm and the
 *      activation quantization before a linear, in one pass;
 *   2. fp8_qk_norm_mrope_cache: fp8_qk_norm_rope_cache with a position on each
 *      of several axes (time, height, width) for images and video;
 *   3. fp8_int4_linear: products with 4-bit weights, a scale and a zero point
 *      for each group of a row (W4A16, "Quantization guide for serving: FP8,
 *      AWQ, GPTQ", the low-batch choice beside W8A8), with fp8_int4_quant_weight
 *      and fp8_int4_pack, which make the weights;
 *   4. fp8_token_logprobs: log probabilities of given tokens, their ranks, the
 *      distributions' entropies and the most likely alternatives.
 *
 * The conventions of fp8w8a8.h hold: device pointers owned by the caller, no
 * allocation, no synchronization, kernels enqueued on `stream`, argument
 * errors returned before anything is enqueued, no output over an input (but
 * where a call says so), bf16 as raw uint16, E4M3 as raw uint8, scales fp32.
 * Results do not depend on timing.
 */
#ifndef FP8W8A8_STEP_H
#define FP8W8A8_STEP_H

#include "fp8w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fp8_add_rms_norm_quant -- residual addition, RMS norm and FP8 quantization.
 *   x        [T, H] bf16, ld_x elements per row                            (input)
 *   residual [T, H] bf16 (ld_r), or NULL: nothing is added                 (input)
 *   residual_out [T, H] bf16 (ld_ro), NULL exactly if residual is; may be
 *            residual itself (same pointer and ld): the stream updated in
 *            place                                                        (output)
 *   weight   [H] bf16                                                       (input)
 *   y        [T, H] bf16 (ld_y), or NULL: the norm without quantization    (output)
 *   q        [T, H] E4M3 codes (ld_q), or NULL: no quantization            (output)
 *   scales   FP8_SCALE_BLOCK: [T, H/128] fp32, ld_s >= H/128               (output)
 *            FP8_SCALE_ROW: scales[t * ld_s], ld_s >= 1                    (output)
 *            FP8_SCALE_TENSOR: not used
 *   scale    FP8_SCALE_TENSOR: one calibrated fp32 in device memory         (input);
 *            the other modes: not used
 *   r = bf16_RNE(x + residual), the sum in fp32 (x itself without a residual),
 *   residual_out = r
 *   v = r / sqrt(mean(r^2) + eps) * weight                        (in fp32)
 *   y = bf16_RNE(v)
 *   q = E4M3_RNE_saturating(v / s), with s = amax / 448 over each 128 values
 *       (FP8_SCALE_BLOCK) or the row (FP8_SCALE_ROW), or s = scale[0]
 * What fp8_block_gemm takes: codes and scales as fp8_quant_act and
 * fp8_quant_act_static lay them out, quantized from the fp32 values (not from
 * y).  A group whose s is 0 (zeros, or an amax below 2^-141, whose 448th part
 * fp32 does not hold) gets codes +-0.  Neither the mean of squares nor its root's
 * reciprocal leaves its range for any finite r; a row of zeros with eps = 0 is NaN
 * (0 / 0).  A NaN in r makes its row NaN, an infinity gives NaN in its place and
 * zeros elsewhere; the codes of a group whose scale is NaN are unspecified.
 * At least one of y and q is given.  H a multiple of 128 up to 65536;
 * eps >= 0; base pointers of x, residual, residual_out, weight, y and q
 * 16-byte aligned, ld of bf16 tensors multiples of 8, ld_q of 16.  scale_mode is
 * not looked at without q.  T == 0 does nothing.  One launch; no workspace. */
fp8_status fp8_add_rms_norm_quant(const uint16_t* x, int64_t ld_x, const uint16_t* residual,
                                  int64_t ld_r, uint16_t* residual_out, int64_t ld_ro,
                                  const uint16_t* weight, float eps, uint16_t* y, int64_t ld_y,
                                  uint8_t* q, int64_t ld_q, float* scales, int64_t ld_s,
                                  int scale_mode, const float* scale, int64_t T, int64_t H,
                                  void* stream);

/* Orders of the axes over the rotated pairs, for fp8_qk_norm_mrope_cache. */
enum { FP8_AXES_SECTIONS = 0, FP8_AXES_IN_TURN = 1 };

/* fp8_qk_norm_mrope_cache -- fp8_qk_norm_rope_cache with positions on several
 * axes: pair i of a head turns by the angle of its axis' position.
 *   positions [A, T] int64, ld_pos elements per axis                       (input)
 *   sections  [A] int64 in HOST memory, read during the call: rotated pairs
 *             of each axis; >= 0, rot_dim / 2 in all                       (input)
 *   axis_order FP8_AXES_SECTIONS: the first sections[0] pairs belong to axis
 *             0, the next sections[1] to axis 1, ...
 *             FP8_AXES_IN_TURN: pair i belongs to axis a = i % A while
 *             i < A * sections[a], else to axis 0; sections of the axes from 1
 *             on must fit, a + A * (sections[a] - 1) < rot_dim / 2
 * 1 <= A <= 4; ld_pos >= T where A > 1.  All else as for fp8_qk_norm_rope_cache; a token with a position
 * outside [0, max_pos) on any axis is padding, also where that axis turns no
 * pair.  With one axis the results are that call's, bit for bit. */
fp8_status fp8_qk_norm_mrope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, int64_t ld_pos, int64_t A, const int64_t* sections, int axis_order,
    const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk, int64_t D, uint16_t* query_out,
    int64_t ld_query_out, uint8_t* key_cache, uint8_t* value_cache, int64_t num_blocks,
    int64_t block_size, const float* k_scale, const float* v_scale, void* stream);

/* Packed 4-bit weights.  8 values of a row, v0 .. v7, take 4 bytes:
 *   byte 0: v0 | v2 << 4   byte 1: v4 | v6 << 4
 *   byte 2: v1 | v3 << 4   byte 3: v5 | v7 << 4
 * (the even values in the lower half word, the odd ones in the upper, so that
 * one mask takes a pair as the matrix unit's operand holds it).  A row of K
 * values is K / 2 bytes, rows are contiguous. */

/* fp8_int4_pack -- packs 4-bit values that a checkpoint holds one a byte.
 *   values [N, K] uint8, ld_v bytes per row, the lower 4 bits of each used  (input)
 *   codes  [N, K / 2] packed                                                (output)
 * K a positive multiple of 128; values 8-byte aligned, ld_v a multiple of 8,
 * codes 16-byte aligned.  N == 0 does nothing. */
fp8_status fp8_int4_pack(const uint8_t* values, int64_t ld_v, uint8_t* codes, int64_t N, int64_t K,
                         void* stream);

/* fp8_int4_quant_weight -- rounds a weight to 4 bits by groups.
 *   w      [N, K] bf16, ld_w elements per row                              (input)
 *   codes  [N, K / 2] packed                                              (output)
 *   scales [N, K / group] fp32, contiguous                                (output)
 *   zeros  [N, K / group] uint8, contiguous, or NULL: symmetric           (output)
 * Per group, with lo = min(min w, 0) and hi = max(max w, 0):
 *   zeros given: s = (hi - lo) / 15, z = min(RNE(-lo / s), 15);
 *   NULL:        s = max(-lo, hi) / 7, z = 8;
 *   code = min(max(RNE(w / s) + z, 0), 15), fp32 divisions.
 * A group whose s is 0 gets codes z (z = 0 where zeros are given).  w and
 * hi - lo are taken to be finite.  Alignment as for fp8_quant_weight_block and
 * fp8_int4_linear.  N == 0 does nothing. */
fp8_status fp8_int4_quant_weight(const uint16_t* w, int64_t ld_w, uint8_t* codes, float* scales,
                                 uint8_t* zeros, int64_t N, int64_t K, int64_t group,
                                 void* stream);

/* Bytes of workspace with which fp8_int4_linear cuts K into runs (0: it does
 * not; nonzero where more than 4 rows of x have too few tiles of the weight for
 * all compute units). */
size_t fp8_int4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* fp8_int4_linear -- out = x . W^T with 4-bit weights.
 *   x      [M, K] bf16, ld_x elements per row                              (input)
 *   codes  [N, K / 2] packed, contiguous                                   (input)
 *   scales [N, K / group] fp32, contiguous                                 (input)
 *   zeros  [N, K / group] uint8, contiguous, or NULL: 8 everywhere         (input)
 *   out    [M, N] bf16, ld_out elements per row                           (output)
 *   out[m, n] = bf16_RNE( sum_g scales[n, g] *
 *                         sum_{k in g} x[m, k] * (code[n, k] - zeros[n, g]) )
 * The matrix unit multiplies bf16 x with the exact integers 16 + code; the sums
 * of a group are fp32, 16 + zero times the group's sum of x is taken off in
 * fp32, and the scaled groups are summed in fp32.  Nothing is rounded below
 * that but the result; where c - z is small the offset's part of the sums makes
 * their rounding up to (16 + c) / |c - z| times as large, and a far value of x with
 * c = z leaves what its products were rounded by.  Where a sum leaves fp32's range on the way (|x| from
 * about 2^112 on), the result is formed again in 64 bits, by a few lanes: right, but
 * slow.  A row of x that holds an infinity or a NaN gives NaN.
 * group 32, 64 or 128; K a positive multiple of 128 below 2^24; any N >= 1 and
 * M >= 0 (M = 0 does nothing); x, codes and scales 16-byte aligned, out 2-byte aligned,
 * ld_x a multiple of 8, ld_out any >= N.  Zeros above 15 are taken as they are.
 * workspace (optional, may be NULL): with at least fp8_int4_workspace_bytes(M,
 * N, K) bytes (16-byte aligned, apart from every tensor of the call, contents
 * not needed and not read afterwards; calls that can overlap need one each) the
 * runs of K that it counts are summed in fp32 by workgroups of their own and
 * then added, in order: the same arithmetic, so results can differ from the
 * uncut call's in the last bits.  A smaller or NULL workspace runs the call
 * uncut.  A row's last bits can depend on M, too, which chooses tiles and runs. */
fp8_status fp8_int4_linear(const uint16_t* x, int64_t ld_x, const uint8_t* codes,
                           const float* scales, const uint8_t* zeros, int64_t group, uint16_t* out,
                           int64_t ld_out, int64_t M, int64_t N, int64_t K, void* workspace,
                           size_t ws_bytes, void* stream);

/* Types of logits. */
enum { FP8_LOGITS_BF16 = 0, FP8_LOGITS_F32 = 1 };

/* Largest k of fp8_token_logprobs. */
#define FP8_MAX_TOP 64

/* Bytes of workspace that fp8_token_logprobs needs (0 where a row's one workgroup
 * does all of it).  The size is that of these T rows, and fewer may need more: many
 * rows of up to 4096 segments of 128 bytes need none, a few are cut into parts.  A buffer
 * for any count up to T has the largest size over 1 .. min(T, 255) and T (from 256
 * rows on it is 0 or grows with T). */
size_t fp8_logprobs_workspace_bytes(int logits_type, int64_t T, int64_t V, int64_t k);

/* fp8_token_logprobs -- what an answer's tokens were worth to the model.
 *   logits [T, V] bf16 or fp32, ld elements per row, any ld >= V           (input)
 *   tokens [T] int64: the token of each row                                (input)
 *   scale  finite, > 0: 1 / temperature; z = scale * logits
 *   logprobs [T] fp32: z[token] - lse                                     (output)
 *   ranks    [T] int32: how many logits of the row are larger             (output)
 *   entropy  [T] fp32: -sum p log p, natural logarithm                    (output)
 *   lse      [T] fp32: log sum exp z                                      (output)
 *   top_logprobs [T, k] fp32, top_ids [T, k] int32, contiguous: the k largest
 *            z - lse, in falling order, of equal logits the lower index first;
 *            both NULL if k is 0                                          (output)
 * One pass over the logits, sums in fp32, in an order that T, V and the row's place
 * in memory choose: last bits can depend on them.  A logit of -inf has probability 0: its log
 * probability is -inf, and it comes among the alternatives after all others.  A log
 * probability below fp32's range is -inf, too, and an lse beyond it an infinity,
 * beside log probabilities as they are.
 * A row of -inf only has lse and log probabilities -inf and entropy 0.  A row
 * with a NaN or +inf is no distribution: its log probabilities, entropy and
 * lse are NaN, its ranks and ids -1.  A token outside [0, V) is padding: log
 * probability 0, rank -1, the row's other outputs as ever.
 * 0 <= k <= min(V, FP8_MAX_TOP); 1 <= V < 2^31; logits aligned to their type;
 * T == 0 does nothing.  workspace: fp8_logprobs_workspace_bytes(...) bytes,
 * 16-byte aligned, contents not needed and not read afterwards; calls that
 * can overlap need one each. */
fp8_status fp8_token_logprobs(const void* logits, int logits_type, int64_t ld,
                              const int64_t* tokens, float scale, int64_t T, int64_t V, int64_t k,
                              float* logprobs, int32_t* ranks, float* entropy, float* lse,
                              float* top_logprobs, int32_t* top_ids, void* workspace,
                              size_t ws_bytes, void* stream);

/* Host-only validation: the argument checks of the calls above, without
 * touching any device.  ws_needed is what the call's *_workspace_bytes gives. */
fp8_status fp8_validate_add_rms_norm_quant(const uint16_t* x, int64_t ld_x,
                                           const uint16_t* residual, int64_t ld_r,
                                           const uint16_t* residual_out, int64_t ld_ro,
                                           const uint16_t* weight, float eps, const uint16_t* y,
                                           int64_t ld_y, const uint8_t* q, int64_t ld_q,
                                           const float* scales, int64_t ld_s, int scale_mode,
                                           const float* scale, int64_t T, int64_t H);
fp8_status fp8_validate_qk_norm_mrope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, int64_t ld_pos, int64_t A, const int64_t* sections, int axis_order,
    const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
    const uint16_t* query_out, int64_t ld_query_out, const uint8_t* key_cache,
    const uint8_t* value_cache, int64_t num_blocks, int64_t block_size, const float* k_scale,
    const float* v_scale);
fp8_status fp8_validate_int4_pack(const uint8_t* values, int64_t ld_v, const uint8_t* codes,
                                  int64_t N, int64_t K);
fp8_status fp8_validate_int4_quant_weight(const uint16_t* w, int64_t ld_w, const uint8_t* codes,
                                          const float* scales, const uint8_t* zeros, int64_t N,
                                          int64_t K, int64_t group);
fp8_status fp8_validate_int4_linear(const uint16_t* x, int64_t ld_x, const uint8_t* codes,
                                    const float* scales, const uint8_t* zeros, int64_t group,
                                    const uint16_t* out, int64_t ld_out, int64_t M, int64_t N,
                                    int64_t K, const void* workspace, size_t ws_bytes);
fp8_status fp8_validate_token_logprobs(const void* logits, int logits_type, int64_t ld,
                                       const int64_t* tokens, float scale, int64_t T, int64_t V,
                                       int64_t k, const float* logprobs, const int32_t* ranks,
                                       const float* entropy, const float* lse,
                                       const float* top_logprobs, const int32_t* top_ids,
                                       const void* workspace, size_t ws_bytes, size_t ws_needed);

#ifdef __cplusplus
}
#endif

#endif /* FP8W8A8_STEP_H */
