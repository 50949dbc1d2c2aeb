/*
 * fp8w8a8_attention.h -- C ABI of the paged FP8 attention step for gfx950.
 *
 * What stands between the FP8 linears of fp8w8a8.h when a model is served
 * from the paged FP8 KV cache (fp8_kv_cache_write / fp8_kv_cache_read):
 *   1. fp8_kv_slot_map: the block tables, cache slots and positions of a
 *      step's tokens, from the requests' lengths;
 *   2. fp8_qk_norm_rope_cache: per-head RMS norm and rotation of queries and
 *      keys, the keys and values stored as E4M3 codes in the same pass;
 *   3. fp8_paged_attention: causal attention over the cache with an optional
 *      sliding window and first tokens that stay visible (sinks);
 *   4. fp8_prefix_attention: the same for a batch whose requests share a
 *      prefix, whose keys and values are read once for all of them.
 * With an fp8 KV-cache dtype keys and values are stored as E4M3, each with
 * its own scale, and restored inside the attention ("FP8 Quantization", D.4;
 * "[vLLM] FP8", KV cache quantization; "Quantization guide for serving: FP8,
 * AWQ, GPTQ", KV-cache FP8 section, 16-token paged blocks).
 *
 * The conventions of fp8w8a8.h hold: device pointers owned by the caller, no
 * allocation, no synchronization, kernels enqueued on `stream`, argument
 * errors returned before anything is enqueued, no output over an input, bf16
 * as raw uint16, E4M3 as raw uint8, scales fp32.  Lengths, offsets and block
 * tables are int32, cache slots and positions int64, all in device memory:
 * no call needs a length on the host, so a step can be captured in a graph.
 * What these arrays hold is checked on the device: no content reaches memory
 * outside the tensors, and what a bad entry means is said at each call.
 */
#ifndef FP8W8A8_ATTENTION_H
#define FP8W8A8_ATTENTION_H

#include "fp8w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fp8_kv_slot_map -- block tables and slot maps of one step.
 *   computed_lens [B] int32: tokens of each request already in the cache (input)
 *   new_lens      [B] int32: tokens that this step adds                   (input)
 *   free_blocks   [num_free] int32: block numbers to hand out, in order   (input)
 *   block_table   [B, table_width] int32, ld_table elements per row: entry i
 *                 is the block of tokens i * block_size ..             (in/out)
 *   slot_mapping, positions  [T] int64                                   (output)
 *   query_offsets [B + 1] int32: first token of each request, then the total
 *   seq_lens      [B] int32: computed + new
 *   blocks_taken  [1] int32: blocks that the step needs
 * Request r keeps its first ceil(computed / block_size) blocks and gets the
 * next ones up to ceil((computed + new) / block_size) from free_blocks, the
 * requests served in order; only those entries of block_table are written.
 * Token i of request r has position computed + i and slot
 *   block * block_size + position % block_size.
 * Negative lengths count as 0.  An entry behind free_blocks' end becomes -1
 * (blocks_taken > num_free says so) and entries behind table_width are not
 * written; tokens without a block (a negative entry, too) get slot -1, which
 * fp8_kv_cache_write and fp8_qk_norm_rope_cache do not store.  Elements of
 * slot_mapping and positions behind the last token are -1.  Sums beyond
 * 2^31 - 1 saturate.  block_size > 0; one launch; no workspace. */
fp8_status fp8_kv_slot_map(const int32_t* computed_lens, const int32_t* new_lens, int64_t B,
                           int64_t block_size, int32_t* block_table, int64_t ld_table,
                           int64_t table_width, const int32_t* free_blocks, int64_t num_free,
                           int64_t* slot_mapping, int64_t* positions, int64_t T,
                           int32_t* query_offsets, int32_t* seq_lens, int32_t* blocks_taken,
                           void* stream);

/* fp8_qk_norm_rope_cache -- norm, rotation and cache store of one step.
 *   query [T, Hq, D], key, value [T, Hk, D] bf16: a token's heads are
 *                 contiguous, tokens ld_* elements apart (slices of one QKV
 *                 row work)                                               (input)
 *   q_weight, k_weight [D] bf16: the norms' weights                        (input)
 *   cos_sin   [max_pos, rot_dim] fp32, contiguous: rot_dim / 2 cosines, then
 *             as many sines, of each position                              (input)
 *   positions, slot_mapping [T] int64                                      (input)
 *   query_out [T, Hq, D] bf16, tokens ld_query_out elements apart         (output)
 *   key_cache, value_cache, num_blocks, block_size, k_scale, v_scale as for
 *             fp8_kv_cache_write                                          (in/out)
 * For a head x of a query or key, with c, s the position's cosines and sines:
 *   y = x / sqrt(mean(x^2) + eps) * weight
 *   (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i)   for i < rot_dim / 2
 * with (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved is
 * nonzero; elements from rot_dim on are only normalized.  Computed in fp32
 * and rounded once: queries to bf16 (round to nearest even; a NaN gives a
 * quiet NaN), keys to E4M3(y / k_scale), values to E4M3(v / v_scale), bit for bit as
 * fp8_kv_cache_write stores them.  A token whose position is outside
 * [0, max_pos) is padding: nothing of it is written.  A slot outside the
 * cache is not stored, its query is written.  Two tokens with one slot leave
 * either token's codes, mixed by head.
 * D a multiple of 16 up to 512, rot_dim a multiple of 16 up to D (0: no
 * rotation, cos_sin may be NULL and max_pos bounds the positions still);
 * base pointers of bf16 tensors, caches and cos_sin 16-byte aligned, ld a
 * multiple of 8.  eps >= 0.  T == 0 does nothing.  No workspace. */
fp8_status fp8_qk_norm_rope_cache(const uint16_t* query, int64_t ld_query, const uint16_t* key,
                                  int64_t ld_key, const uint16_t* value, int64_t ld_value,
                                  const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                  const float* cos_sin, int64_t max_pos, int64_t rot_dim,
                                  int interleaved, const int64_t* positions,
                                  const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk,
                                  int64_t D, uint16_t* query_out, int64_t ld_query_out,
                                  uint8_t* key_cache, uint8_t* value_cache, int64_t num_blocks,
                                  int64_t block_size, const float* k_scale, const float* v_scale,
                                  void* stream);

/* Bytes of workspace that fp8_paged_attention (shared_prefix = 0) or
 * fp8_prefix_attention (nonzero) needs for T query tokens in B requests on
 * the current device.  It grows with T and may shrink as B grows: what (T, 1)
 * needs is enough for T tokens in any number of requests. */
size_t fp8_attention_workspace_bytes(int shared_prefix, int64_t T, int64_t B, int64_t Hq,
                                     int64_t Hk, int64_t D);

/* fp8_paged_attention -- attention of a ragged batch over the paged FP8 cache.
 *   query [T, Hq, D] bf16, tokens ld_query elements apart                  (input)
 *   key_cache, value_cache [num_blocks, block_size, Hk, D] E4M3           (input)
 *   block_table [B, table_width] int32, ld_table elements per row          (input)
 *   seq_lens    [B] int32: cached tokens of each request, the step's own
 *               among them                                                 (input)
 *   query_offsets [B + 1] int32: request r's queries are tokens
 *               query_offsets[r] .. query_offsets[r + 1] - 1, its last     (input)
 *   k_scale, v_scale  one fp32 each in device memory                       (input)
 *   out   [T, Hq, D] bf16, tokens ld_out elements apart                   (output)
 *   lse   [T, Hq] fp32, contiguous, or NULL                               (output)
 * Query i of n in a request of length L stands at position p = L - n + i.
 * Its head h reads KV head h / (Hq / Hk):
 *   s_j = scale * k_scale * <q, dec(key_j)>  over the visible j:
 *         j <= p and (window == 0 or p - j < window or j < sinks)
 *   out = bf16( v_scale * sum_j exp(s_j) dec(value_j) / sum_j exp(s_j) )
 *   lse = log sum_j exp(s_j)
 * The products <q, key> are exact with fp32 sums; scores, maxima, sums and
 * outputs are held in fp32; exp(s_j) is rounded to fp16 for the product with
 * the values, not for the sum below it: to 11 bits, and to a multiple of 2^-34
 * of the row's largest where it is below 2^-24 of that.  Where the scores of a
 * row pass 2^20 they are rounded to fp32 before the maximum is subtracted.
 * A query that sees no key (L = 0, p < 0, or only unmapped pages) gets zeros
 * and lse = -inf.  A key in a page that the table does not map (an entry
 * outside [0, num_blocks), or behind table_width) is not visible, nor is one
 * at 2^31 - 65536 or behind it in its request or prefix.  Codes in
 * places that a query does not see, NaN among them, do not reach it.  Rows
 * of out and lse in no request's range are left as they were.  Offsets are
 * clamped to [0, T] and should be nondecreasing.
 * D 64, 128 or 256; Hq a multiple of Hk; window, sinks >= 0 (sinks without a
 * window change nothing); num_blocks * block_size < 2^31; T * Hq < 2^31.  The
 * result does not depend on timing.
 * workspace: fp8_attention_workspace_bytes(0, T, B, Hq, Hk, D) bytes, 16-byte
 * aligned, contents not needed and not read afterwards; calls that can
 * overlap need one each. */
fp8_status fp8_paged_attention(const uint16_t* query, int64_t ld_query, const uint8_t* key_cache,
                               const uint8_t* value_cache, int64_t num_blocks, int64_t block_size,
                               const int32_t* block_table, int64_t ld_table, int64_t table_width,
                               const int32_t* seq_lens, const int32_t* query_offsets, int64_t B,
                               const float* k_scale, const float* v_scale, float scale,
                               int64_t window, int64_t sinks, uint16_t* out, int64_t ld_out,
                               float* lse, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                               void* workspace, size_t ws_bytes, void* stream);

/* fp8_prefix_attention -- fp8_paged_attention (window 0) for a batch whose
 * requests all start with the same prefix_len[0] tokens:
 *   prefix_table [prefix_width] int32: the prefix's blocks (NULL if the width
 *                is 0)                                                     (input)
 *   prefix_len   [1] int32 in device memory; the prefix may end inside a
 *                block                                                     (input)
 *   block_table, seq_lens describe what follows the prefix in each request
 *   (token 0 of a request's own blocks is position prefix_len).
 * Every query sees the whole prefix and its own request's keys up to itself.
 * Where a request has seq_lens[r] >= n - 1 for its n queries, that is the
 * result of fp8_paged_attention over the joined tokens, up to the order of
 * the fp32 sums.  With fewer own tokens the first n - 1 - seq_lens[r] queries
 * are tokens inside the prefix, and they see all of it nevertheless, also the
 * keys behind themselves: to run a part of the prefix itself causally, call
 * fp8_paged_attention over the joined tokens.  The prefix is read once for
 * groups of queries of all requests together.  A negative prefix_len counts
 * as 0; unmapped pages of either table are not visible.  Rows in no request's range are left as
 * they were.  workspace: fp8_attention_workspace_bytes(1, ...) bytes. */
fp8_status fp8_prefix_attention(const uint16_t* query, int64_t ld_query, const uint8_t* key_cache,
                                const uint8_t* value_cache, int64_t num_blocks, int64_t block_size,
                                const int32_t* prefix_table, int64_t prefix_width,
                                const int32_t* prefix_len, const int32_t* block_table,
                                int64_t ld_table, int64_t table_width, const int32_t* seq_lens,
                                const int32_t* query_offsets, int64_t B, const float* k_scale,
                                const float* v_scale, float scale, uint16_t* out, int64_t ld_out,
                                float* lse, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                void* workspace, size_t ws_bytes, void* stream);

/* Host-only validation: the argument checks of the calls above, without
 * touching any device. */
fp8_status fp8_validate_kv_slot_map(const int32_t* computed_lens, const int32_t* new_lens,
                                    int64_t B, int64_t block_size, const int32_t* block_table,
                                    int64_t ld_table, int64_t table_width,
                                    const int32_t* free_blocks, int64_t num_free,
                                    const int64_t* slot_mapping, const int64_t* positions,
                                    int64_t T, const int32_t* query_offsets,
                                    const int32_t* seq_lens, const int32_t* blocks_taken);
fp8_status fp8_validate_qk_norm_rope_cache(
    const uint16_t* query, int64_t ld_query, const uint16_t* key, int64_t ld_key,
    const uint16_t* value, int64_t ld_value, const uint16_t* q_weight, const uint16_t* k_weight,
    float eps, const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
    const int64_t* positions, const int64_t* slot_mapping, int64_t T, int64_t Hq, int64_t Hk,
    int64_t D, const uint16_t* query_out, int64_t ld_query_out, const uint8_t* key_cache,
    const uint8_t* value_cache, int64_t num_blocks, int64_t block_size, const float* k_scale,
    const float* v_scale);
/* prefix_table and prefix_len both NULL with prefix_width 0: the checks of
 * fp8_paged_attention; else those of fp8_prefix_attention.  ws_needed is
 * what fp8_attention_workspace_bytes gives (that call asks the device). */
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
                                  size_t ws_bytes, size_t ws_needed);

#ifdef __cplusplus
}
#endif

#endif /* FP8W8A8_ATTENTION_H */
