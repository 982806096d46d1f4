/*
 * kv_cache.h -- C ABI of serving with a paged cache of keys and values by head,
 * in the same library (libidx_paged_mqa.so): the page tables and slot maps of a
 * batch, built from its requests' lengths; the store of new keys and values; the
 * bounds of each page's keys and a query's score of a page by them, which
 * idx_topk_logits selects pages from; and the attention of one new token per row
 * over all its pages or the selected ones.
 *
 * Everything paged_mqa_logits.h says of ownership, threading, streams, errors
 * and device data holds here too: device pointers owned by the caller, no
 * state, no allocation, no host synchronisation, arguments validated on the
 * host, nothing launched unless the status is IDX_OK.  The grids depend on
 * the scalar arguments alone, so every call can be captured into a HIP graph.
 *
 * The cache.  Pools of pages of 64 positions, one of keys and one of values, of
 * kv_heads heads of head_dim (64, 128 or 256) values.  Head h of page g is a
 * block at k_pages + g*kv_page_stride + h*kv_head_stride (bytes), its values at
 * v_pages with the same strides:
 *   fp8   [64][head_dim] e4m3fn codes, position major; the fp32 scale of slot i
 *         at kscale + g*kscale_page_stride + h*kscale_head_stride + 4*i (bytes),
 *         and at vscale
 *   bf16  [64][head_dim] bf16
 * so that head h of the keys is a pool of paged_mqa_logits.h and latent_cache.h
 * itself, with its base h*kv_head_stride further on.  In any order: the strides
 * are at least a block's bytes (fp8 64*head_dim, bf16 128*head_dim; scales 256)
 * and multiples of 16 (scales 4), the page strides at most 2^32, the head strides
 * at most 2^38 (not looked at if kv_heads is 1); k_pages and v_pages are 16-byte
 * aligned, the scales 4-byte.
 */
#ifndef IDX_KV_CACHE_H
#define IDX_KV_CACHE_H

#include "latent_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The page tables and slot maps of a step, from the lengths of its requests.
 * Request r has cached[r] positions and gets added[r] more (negative lengths
 * count as 0).  With
 *
 *   low_r  = ceil(cached[r] / 64),  high_r = ceil((cached[r] + added[r]) / 64), at most table_width
 *   base_r = sum_{s<r} max(0, high_s - low_s)
 *
 * its new pages are free_pages[base_r ..): page_table[r][j] = free_pages[base_r
 * + j - low_r] for low_r <= j < high_r, -1 where the list is too short; its other
 * entries are left as they are.  The new tokens, request by request, are the
 * batch's first rows; token i of request r, row t = i + sum_{s<r} added[s]:
 *
 *   positions[t] = p = cached[r] + i
 *   slots[t]     = 64 * page_table[r][p / 64] + p % 64; -1 where that page is
 *                  negative or past the table
 *   row_table[t] = r                                       seqlens[t] = p + 1
 *
 * (at most 2^31 - 1).  Rows t < n past the last token are padding: slot -1, position
 * 0, row_table 0, seqlens 0; tokens past the n-th get no row (their pages are handed
 * out all the same).
 *
 *   cached, added  int32 [requests], 4-byte aligned; requests in [0, 65536].
 *   free_pages     int32 [num_free], 4-byte aligned; may be NULL if num_free is 0.
 *   page_table     int32, 4-byte aligned, request r's at page_table +
 *                  r*page_table_row_stride (elements, >= table_width where there
 *                  is more than one request); may be NULL if table_width is 0.
 *   n              rows of the outputs, >= 0.
 *   slots, positions    int64 [n], 8-byte aligned, or NULL: not written.
 *   row_table, seqlens  int32 [n], 4-byte aligned, or NULL.
 *   starts         int64 [requests + 1], or NULL: the first row of each request,
 *                  and the number of tokens (which may be above n).
 *   taken          int64 [1], or NULL: the pages asked for (above num_free: the
 *                  list was too short).
 * The arrays do not overlap.
 */
int idx_plan_batch(const int32_t* cached, const int32_t* added, int32_t requests, const int32_t* free_pages,
                   int64_t num_free, int32_t* page_table, int32_t table_width, int64_t page_table_row_stride,
                   int64_t n, int64_t* slots, int64_t* positions, int32_t* row_table, int32_t* seqlens,
                   int64_t* starts, int64_t* taken, hipStream_t stream);

/*
 * Paged store of keys and values: token t's kv_heads vectors of each go to slot
 * slots[t] (page slots[t] / 64, position slots[t] % 64), quantised vector by
 * vector as idx_store_keys_fp8 does it:
 *
 *   scale   = amax > 0 ? amax / 448 : 1        amax = max_d |x_d|
 *   code_d  = e4m3fn(clamp(x_d / scale, -448, 448)), round to nearest even
 *
 * A NaN has no part in amax; a quotient that is NaN becomes +-448 with the sign of
 * x_d.  A slot outside [0, 64*num_pages) -- e.g. -1 for a padding token -- skips its
 * token.  Two tokens with the same slot race.
 *
 *   keys, values   bf16, head h of token t at keys + t*k_row_stride + h*head_dim
 *                  (elements); 16-byte aligned, the strides multiples of 8 and
 *                  >= kv_heads*head_dim.
 *   slots          int64 [n], 8-byte aligned.
 *   n, kv_heads    >= 0; 0 returns IDX_OK with no launch.
 */
int idx_store_kv_fp8(const void* keys, const void* values, const int64_t* slots, int64_t n, int32_t kv_heads,
                     int32_t head_dim, int64_t k_row_stride, int64_t v_row_stride, void* k_pages, void* v_pages,
                     float* kscale, float* vscale, int64_t num_pages, int64_t kv_page_stride,
                     int64_t kv_head_stride, int64_t kscale_page_stride, int64_t kscale_head_stride,
                     hipStream_t stream);

/* bf16 counterpart: a copy. */
int idx_store_kv_bf16(const void* keys, const void* values, const int64_t* slots, int64_t n, int32_t kv_heads,
                      int32_t head_dim, int64_t k_row_stride, int64_t v_row_stride, void* k_pages, void* v_pages,
                      int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride, hipStream_t stream);

/*
 * Bounds of pages' keys: for row b and every page j with first[b] / 64 <= j <
 * ceil(L_b / 64), L_b = clamp(seqlens[b], 0, table_width * 64), of id g =
 * page_table_b[j], and every head h
 *
 *   bounds[g][h][0][d] = min_i k_i[d]     bounds[g][h][1][d] = max_i k_i[d]
 *
 * over the page's positions i below L_b, those before first[b] among them, k_i the
 * float32 product of code and scale (or the bf16 value), rounded to bf16 outwards
 * (bf16 keys: exact).  A NaN has no part in them (a dim of nothing else: 0 and 0);
 * beyond bf16's largest finite value (infinities) they are that value.  After a
 * prefill first is 0 (or NULL), after a decode step the row's length before it.  A
 * page id outside [0, num_pages) skips its page; a page that two rows name races
 * unless they agree on its positions.
 *
 *   k_pages, kscale, num_pages, strides   as above.
 *   page_table, row_table, num_tables, page_table_row_stride
 *              row b's table as in idx_latent_attention_fp8; a row_table index
 *              outside [0, num_tables) skips its row.
 *   first      int32 [rows], 4-byte aligned, or NULL: 0 for all (a negative one too).
 *   seqlens    int32 [rows], 4-byte aligned.
 *   bounds     bf16 [num_pages][kv_heads][2][head_dim], 16-byte aligned.
 *   rows * ceil(kv_heads / 4) less than 2^24.
 */
int idx_page_bounds_fp8(const void* k_pages, const float* kscale, const int32_t* page_table,
                        const int32_t* row_table, int32_t num_tables, const int32_t* first,
                        const int32_t* seqlens, void* bounds, int32_t rows, int32_t kv_heads, int32_t head_dim,
                        int32_t table_width, int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                        int64_t kscale_page_stride, int64_t kscale_head_stride, int64_t page_table_row_stride,
                        hipStream_t stream);

/* bf16 counterpart (no scales). */
int idx_page_bounds_bf16(const void* k_pages, const int32_t* page_table, const int32_t* row_table,
                         int32_t num_tables, const int32_t* first, const int32_t* seqlens, void* bounds,
                         int32_t rows, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                         int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                         int64_t page_table_row_stride, hipStream_t stream);

/*
 * Scores of pages: the most that any key within a page's bounds could score with
 * any of the num_heads / kv_heads query heads of a key head,
 *
 *   scores[b][h][j] = max_{i in group h} sum_d max(q_bi[d] lo_gh[d], q_bi[d] hi_gh[d])    j < C_b
 *                     -inf                                                                j >= C_b
 *
 * with C_b = ceil(L_b / 64) live pages, L_b as above, g = page_table_b[j], lo and hi
 * the bounds of idx_page_bounds (lo <= hi); +inf for the first first_pages and the
 * last last_pages of the live ones, which so are selected first.  Group h is the heads
 * h*G .. h*G + G - 1, G = num_heads / kv_heads.  Sums are float32; a NaN among q or
 * the bounds makes the score NaN, an infinity may.  A page id outside [0, num_pages), or a table index
 * outside [0, num_tables), scores NaN (a page of the first or last ones +inf).
 * page_counts[b][h] = C_b: scores and counts are what idx_topk_logits takes (rows *
 * kv_heads rows of table_width columns), and what it selects is the page_idx of
 * idx_kv_attention.
 *
 *   q            bf16 [rows][num_heads][head_dim], contiguous, 16-byte aligned.
 *   bounds       as above.
 *   scores       fp32, row (b, h) at scores + (b*kv_heads + h)*score_stride
 *                (elements, >= table_width); 4-byte aligned.  Every element below
 *                table_width is written.
 *   page_counts  int32 [rows][kv_heads], 4-byte aligned, or NULL.
 *   num_heads    a multiple of kv_heads, at most 128 * kv_heads; 0 returns IDX_OK with
 *                no launch.
 *   first_pages, last_pages   >= 0.
 */
int idx_page_scores(const void* q, const void* bounds, const int32_t* page_table, const int32_t* row_table,
                    int32_t num_tables, const int32_t* seqlens, float* scores, int32_t* page_counts,
                    int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                    int64_t num_pages, int64_t page_table_row_stride, int64_t score_stride, int32_t first_pages,
                    int32_t last_pages, hipStream_t stream);

/*
 * Attention of one new token per row over the paged keys and values.  Row b is a
 * query of num_heads heads; head i reads key head h = i / (num_heads / kv_heads):
 *
 *   L_b      = clamp(seqlens[b], 0, table_width * 64),  C_b = ceil(L_b / 64)
 *   S_bh     = positions p < L_b of the pages p / 64 among the first min(k, C_b)
 *              entries of page_idx[b][h] -- what idx_topk_logits leaves; an
 *              entry outside [0, C_b) is skipped, one that is there twice counts
 *              twice -- or every p < L_b if k is -1
 *   x_ip     = scale * <q[b][i], k_p>
 *   z_i      = sum_{p in S_bh} exp(x_ip) (+ exp(sinks[i]))
 *   out[b][i] = sum_{p in S_bh} exp(x_ip) v_p / z_i          lse[b][i] = ln z_i
 *
 * A row with nothing in S_bh and no sink gets out 0 and lse -inf.  Two results over
 * disjoint sets of positions (a sink in one of them at most) join as
 * (out1 e^lse1 + out2 e^lse2) / (e^lse1 + e^lse2).  Slots at or past L_b have no part
 * in the result, whatever they hold.  A page of S_bh whose id lies outside [0,
 * num_pages), or whose row's table index lies outside [0, num_tables), is not read:
 * it makes out and lse of the group's heads NaN.  Scores, sums and outputs are
 * float32 until the one rounding of out, scores times log2(e) (beyond +-2.35e38 they
 * are infinite); the probability of a position (times the value's e4m3 scale) enters
 * its product with v_p rounded to 16 bits (two bf16) where at most 16 query heads
 * share a key head, to bf16 where more do.
 *
 *   q          bf16 [rows][num_heads][head_dim], contiguous, 16-byte aligned.
 *   page_table, row_table, num_tables, page_table_row_stride
 *              as in idx_latent_attention_fp8 (a stride of 0: one table).
 *   page_idx   int32 [rows][kv_heads][k], 4-byte aligned; NULL if k is -1 (it may
 *              be if k is 0).
 *   seqlens    int32 [rows], 4-byte aligned.
 *   sinks      fp32 [num_heads], 4-byte aligned, or NULL.
 *   out        bf16 [rows][num_heads][head_dim], 16-byte aligned.
 *   lse        fp32 [rows][num_heads], 4-byte aligned, or NULL.
 *   num_heads  a multiple of kv_heads, at most 128 * kv_heads; rows * num_heads at
 *              most 8,000,000.
 *   k >= -1.   scale * log2(e) finite.
 *   workspace  idx_kv_attention_workspace(...) bytes on the call's device, 16-byte
 *              aligned; NULL where that is 0.  It holds nothing between calls, but
 *              calls that may run at the same time (captured ones included) need
 *              one each.
 */
int idx_kv_attention_fp8(const void* q, const void* k_pages, const void* v_pages, const float* kscale,
                         const float* vscale, const int32_t* page_table, const int32_t* row_table,
                         int32_t num_tables, const int32_t* page_idx, const int32_t* seqlens,
                         const float* sinks, void* out, float* lse, int32_t rows, int32_t num_heads,
                         int32_t kv_heads, int32_t head_dim, int32_t table_width, int64_t num_pages,
                         int64_t kv_page_stride, int64_t kv_head_stride, int64_t kscale_page_stride,
                         int64_t kscale_head_stride, int64_t page_table_row_stride, int32_t k, float scale,
                         void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* bf16 counterpart (no scales). */
int idx_kv_attention_bf16(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                          const int32_t* row_table, int32_t num_tables, const int32_t* page_idx,
                          const int32_t* seqlens, const float* sinks, void* out, float* lse, int32_t rows,
                          int32_t num_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                          int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                          int64_t page_table_row_stride, int32_t k, float scale, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that a call of these sizes needs on the current device (0:
 * none; -1: sizes out of range). */
int64_t idx_kv_attention_workspace(int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                   int32_t table_width, int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* IDX_KV_CACHE_H */
