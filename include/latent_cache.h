/*
 * latent_cache.h -- C ABI of the operators around the indexer, in the same
 * library (libidx_paged_mqa.so): the norm and rotation of queries, the norm,
 * rotation and paged store of keys and latents, the read back of stored
 * slots, and the attention over the positions that the top-k selected.
 *
 * Everything paged_mqa_logits.h says of ownership, threading, streams, errors
 * and device data holds here too: device pointers owned by the caller, no
 * state, no allocation, no host synchronisation, arguments validated on the
 * host, nothing launched unless the status is IDX_OK.  The grids depend on
 * the scalar arguments alone, so every call can be captured into a HIP graph.
 *
 * The paged cache.  A pool of pages of 64 positions, D values a position: 128
 * for index keys, 512 for the attention's latents ("The Dispatch Decision:
 * Wiring a Triton Kernel into Production", section "The Problem That Led
 * Here": the fused norm + rotation + store kernel takes head_dim 128 besides
 * 512).  Pages are laid out as the indexer's:
 *   fp8   [64][D] e4m3fn codes, position major, and one fp32 scale a position
 *         (64 of them a page, right behind the codes in the fused block of
 *         64*D + 256 bytes, or in a buffer of their own);
 *   bf16  [64][D] bf16.
 */
#ifndef IDX_LATENT_CACHE_H
#define IDX_LATENT_CACHE_H

#include "paged_mqa_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values of a latent vector: key and value of its position at once. */
#define IDX_LATENT_DIM 512

/* Flags of the norm and rotation. */
#define IDX_NORM_OFF 1u     /* no norm and no weight: the vectors are only rotated */
#define IDX_ROPE_LEADING 2u /* the first rope_dim values are rotated, not the last */
#define IDX_ROPE_HALVES 4u  /* pairs (j, j + rope_dim/2), not neighbours (2j, 2j + 1) */

/*
 * Norm and rotation of vectors, head by head, in one pass:
 *
 *   y      = x / sqrt(mean(x^2) + eps) * norm_weight
 *   theta  = position * inv_freq[j]                       j < rope_dim / 2
 *   (a, b) <- (a cos(theta) - b sin(theta), a sin(theta) + b cos(theta))
 *
 * for the pairs (a, b) of the rope_dim rotated values of y, the rest of y as
 * it is.  Everything in float32 but the angle, whose product and reduction are
 * in float64 (inv_freq's fp32 values taken as exact): theta is off by at most
 * |theta| 2^-51 + 2^-25, and nothing is left of angles from 2^51 on but that the
 * rotation is one.  One rounding to bf16 at the end.  A negated inv_freq turns a
 * rotation back; one that is NaN or infinite makes its pairs NaN.
 *
 *   x            bf16, vector h of token t at x + t*x_row_stride + h*head_dim
 *                (elements); 16-byte aligned, x_row_stride a multiple of 8 and
 *                >= num_heads*head_dim.
 *   norm_weight  fp32 [head_dim], 16-byte aligned; NULL: all ones.  Must be
 *                NULL with IDX_NORM_OFF.
 *   positions    int64 [n], 8-byte aligned; any value whose float64 is exact
 *                (|p| <= 2^53).  May be NULL if rope_dim is 0.
 *   inv_freq     fp32 [rope_dim/2], 4-byte aligned.  May be NULL if rope_dim
 *                is 0.
 *   out          bf16 [n][num_heads][head_dim], contiguous, 16-byte aligned.
 *                May be x itself where x is contiguous too; no other overlap.
 *   n, num_heads >= 0; 0 returns IDX_OK with no launch.
 *   head_dim     64, 128, 256 or 512.
 *   rope_dim     a multiple of 16 in [0, head_dim].
 *   eps          finite and >= 0.
 */
int idx_norm_rope(const void* x, const float* norm_weight, const int64_t* positions,
                  const float* inv_freq, void* out, int64_t n, int32_t num_heads, int32_t head_dim,
                  int32_t rope_dim, uint32_t flags, float eps, int64_t x_row_stride,
                  hipStream_t stream);

/*
 * Norm, rotation and paged store in one pass: the vectors of n tokens (one
 * each) are normed and rotated as above, quantised from their float32 values
 *
 *   scale  = amax > 0 ? amax / 448 : 1                    amax = max_d |y_d|
 *   code_d = e4m3fn(clamp(y_d / scale, -448, 448)), round to nearest even
 *
 * and written to their slots: the quantiser of idx_store_keys_fp8 over
 * head_dim values (with IDX_NORM_OFF and rope_dim 0 the bytes are the same).  The
 * norm's factor 1 / sqrt(mean(x^2) + eps), which the quotients do not depend on,
 * may be applied to the scale instead of the values: scale and quotients are the
 * formula's but for the order of their float32 roundings, and a code beside a
 * rounding border may be the other one.  A token's bytes depend on its own
 * arguments alone, not on the tokens beside it.  A NaN has no part in amax; a
 * quotient that is NaN becomes +-448 with the sign of y_d.
 * Arguments as idx_norm_rope and idx_store_keys_fp8 except:
 *   head_dim     128 (index keys) or 512 (latents).
 *   kv_page_stride  bytes, >= 64*head_dim, multiple of 16.
 * A slot outside [0, 64*num_pages) -- e.g. -1 for a padding token -- skips its
 * token.  Two tokens with the same slot race.
 */
int idx_norm_rope_store_fp8(const void* x, const float* norm_weight, const int64_t* positions,
                            const float* inv_freq, const int64_t* slots, int64_t n, int32_t head_dim,
                            int32_t rope_dim, uint32_t flags, float eps, int64_t x_row_stride,
                            void* kv_pages, float* kscale, int64_t num_pages, int64_t kv_page_stride,
                            int64_t kscale_page_stride, hipStream_t stream);

/* bf16 counterpart: the float32 values are rounded to bf16; kv_page_stride >=
 * 128*head_dim, no scales. */
int idx_norm_rope_store_bf16(const void* x, const float* norm_weight, const int64_t* positions,
                             const float* inv_freq, const int64_t* slots, int64_t n, int32_t head_dim,
                             int32_t rope_dim, uint32_t flags, float eps, int64_t x_row_stride,
                             void* kv_pages, int64_t num_pages, int64_t kv_page_stride,
                             hipStream_t stream);

/*
 * Read back of stored slots: out[t] = bf16(code * scale) of slot slots[t]
 * (fp8: the float32 product rounded to nearest even) or its bf16 values.  The
 * row of a slot outside [0, 64*num_pages) is left as it was, as its token was
 * skipped by the store.  A slot may be read any number of times.
 *   slots      int64 [n], 8-byte aligned.
 *   head_dim   128 or 512.
 *   out        bf16, row t at out + t*out_row_stride (elements), 16-byte
 *              aligned; out_row_stride a multiple of 8 and >= head_dim.
 */
int idx_load_slots_fp8(const void* kv_pages, const float* kscale, const int64_t* slots, int64_t n,
                       int32_t head_dim, int64_t num_pages, int64_t kv_page_stride,
                       int64_t kscale_page_stride, void* out, int64_t out_row_stride,
                       hipStream_t stream);

/* bf16 counterpart (no scales). */
int idx_load_slots_bf16(const void* kv_pages, const int64_t* slots, int64_t n, int32_t head_dim,
                        int64_t num_pages, int64_t kv_page_stride, void* out, int64_t out_row_stride,
                        hipStream_t stream);

/*
 * Attention over the paged latents.  Row b is one query token of num_heads
 * heads; S_b are the positions it attends to; position p = 64*j + i has the
 * latent c_p (code * scale, or its bf16 values) of slot i of page
 * page_table_b[j], key and value of every head:
 *
 *   L_b      = clamp(seqlens[b], 0, table_width * 64)
 *   S_b      = the entries p, 0 <= p < L_b, among the first min(k, L_b) of
 *              topk_idx[b] -- what idx_topk_logits leaves; other entries are
 *              skipped, one that is there twice counts twice --
 *              or every p < L_b if k is -1
 *   x_hp     = scale * <q[b][h], c_p>
 *   z_h      = sum_{p in S_b} exp(x_hp) (+ exp(sinks[h]))
 *   out[b][h] = sum_{p in S_b} exp(x_hp) c_p / z_h          lse[b][h] = ln z_h
 *
 * A row with nothing in S_b and no sink gets out 0 and lse -inf.  Two results
 * over disjoint sets of positions (a sink in one of them at most) join as
 * (out1 e^lse1 + out2 e^lse2) / (e^lse1 + e^lse2).  Slots that no position of
 * S_b names are not read, whatever they hold.  A position of S_b whose page id
 * lies outside [0, num_pages), or whose row's table index lies outside
 * [0, num_tables), is not read either: it makes its row's out and lse NaN.
 * Scores, sums and outputs are float32 until the one rounding of out; the
 * probability of a position is rounded to bf16 for its product with c_p.
 *
 *   q          bf16 [rows][num_heads][512], contiguous, 16-byte aligned.
 *   kv_pages, kscale, num_pages, kv_page_stride, kscale_page_stride
 *              the pool of 512-value pages: kv_page_stride >= 32768 bytes
 *              (bf16: 65536), the rest as in idx_paged_mqa_logits_fp8.
 *   page_table int32, 4-byte aligned: row b's table (table_width entries) at
 *              page_table + t*page_table_row_stride with t = b, or
 *              t = row_table[b] where row_table is not NULL.  A stride of 0
 *              gives every row one table.
 *   row_table  int32 [rows] or NULL, 4-byte aligned; num_tables >= 0 is read
 *              with it only.
 *   topk_idx   int32 [rows][k], 4-byte aligned; NULL if k is -1 (it may be if k
 *              is 0).
 *   seqlens    int32 [rows], 4-byte aligned.
 *   sinks      fp32 [num_heads], 4-byte aligned, or NULL.
 *   out        bf16 [rows][num_heads][512], 16-byte aligned.
 *   lse        fp32 [rows][num_heads], 4-byte aligned, or NULL.
 *   rows, num_heads   >= 0; 0 returns IDX_OK with no launch.  num_heads at most
 *              128; rows times blocks of 64 heads at most 8,000,000.
 *   head_dim   must be 512.
 *   table_width >= 0, at most 16,777,216 (page_table may be NULL if it is 0).
 *   k >= -1.   scale * log2(e) finite.
 *   workspace  idx_latent_attention_workspace(rows, num_heads, table_width, k)
 *              bytes on the call's device, 16-byte aligned; NULL where that is
 *              0.  It holds nothing between calls, but calls that may run at the
 *              same time (captured ones included) need one each.
 */
int idx_latent_attention_fp8(const void* q, const void* kv_pages, const float* kscale,
                             const int32_t* page_table, const int32_t* row_table, int32_t num_tables,
                             const int32_t* topk_idx, const int32_t* seqlens, const float* sinks,
                             void* out, float* lse, int32_t rows, int32_t num_heads, int32_t head_dim,
                             int32_t table_width, int64_t num_pages, int64_t kv_page_stride,
                             int64_t kscale_page_stride, int64_t page_table_row_stride, int32_t k,
                             float scale, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream);

/* bf16 counterpart (no scales). */
int idx_latent_attention_bf16(const void* q, const void* kv_pages, const int32_t* page_table,
                              const int32_t* row_table, int32_t num_tables, const int32_t* topk_idx,
                              const int32_t* seqlens, const float* sinks, void* out, float* lse,
                              int32_t rows, int32_t num_heads, int32_t head_dim, int32_t table_width,
                              int64_t num_pages, int64_t kv_page_stride,
                              int64_t page_table_row_stride, int32_t k, float scale, void* workspace,
                              int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that a call of these sizes needs on the current device (0:
 * none; -1: sizes out of range). */
int64_t idx_latent_attention_workspace(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* IDX_LATENT_CACHE_H */
