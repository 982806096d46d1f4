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
 * in float64 (inv_freq's fp32 values taken as exact), and one rounding to bf16
 * at the end.  A negated inv_freq turns a rotation back.
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
 * head_dim values (with IDX_NORM_OFF and rope_dim 0 the bytes are the same).
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

#ifdef __cplusplus
}
#endif

#endif /* IDX_LATENT_CACHE_H */
