/*
 * dspark_draft_step.h -- C ABI of what a serving loop does around the target's
 * run over the drafted tokens: their verification against the target's
 * probabilities, the accepted path's K/V moved behind the context, the pages
 * of the pool shared, copied, reserved and freed, and a cache of 8-bit codes
 * whose scale follows the data, one per page and head: its insert and the
 * attention that reads it.  None of it needs a length on the host, so a whole
 * step can be captured into a CUDA graph.
 *
 * Caches, block tables and conventions are those of dspark_draft_attn.h: the
 * caller owns every buffer, the functions allocate, synchronise and copy
 * nothing, return a dspark_status and never throw; what device memory holds
 * out of range is never dereferenced and raises a bit in *error_flags (NULL:
 * unreported).  A page is a block of the cache: block_size tokens of every
 * head, in every layer.
 *
 * Page-scaled caches.  kv_dtype DSPARK_KV_FP8_E4M3 with block_scales, device
 * int8 [num_blocks, num_kv_heads, 2]: the K (entry 0) or V (entry 1) that a
 * code c of a page and head stands for is e4m3(c) * 2^scale.  Scales lie in
 * [-32, 31]; others are taken as the nearer end.  With a power of two no code
 * loses a bit when a page's scale grows, except those that become subnormal.
 */
#ifndef DSPARK_DRAFT_STEP_H
#define DSPARK_DRAFT_STEP_H

#include "dspark_draft_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSPARK_FLAG_PAGES 0x40u /* fewer free pages than asked for: the request (or pair) is left as it was */
#define DSPARK_FLAG_ROW 0x80u   /* a row of probabilities without any, or a token or parent out of range */
#define DSPARK_FLAG_REFS 0x100u /* a page given back that nobody held */

/*
 * dspark_verify_drafts -- which drafted tokens the target accepts, and the
 * token behind them, distributed as the target's own.
 *
 * Request b's rows are [row_start[b], row_start[b + 1]) of the inputs.  Its row
 * 0 is the last accepted token, row i >= 1 a drafted token that was drawn
 * behind row parents[i] < i (NULL: behind row i - 1, a chain).  Row r of
 * `target` (`draft`) is the target's (drafter's) distribution of the token
 * behind row r.  From row 0 on, the children of the row reached are tested in
 * row order: with R_0 = p, Z_0 = 1, child x is accepted where
 *   u_x q_k(x) Z_k < R_k(x),
 * else R_{k+1} = max(R_k - Z_k q_k, 0), Z_{k+1} = sum R_{k+1}.  q_k is q
 * (replacement 1: each child was drawn from all of it), or q without the
 * children rejected before, divided by what is left (replacement 0: a row's
 * children are distinct).  draft NULL: the drafter takes its tokens without
 * drawing; q_k is 1 at the child, R_{k+1} is R_k without it and Z_{k+1} = Z_k -
 * R_k(x).  An accepted child is the next row reached; where none is, or after
 * max_accepted tokens, the last token is the first i for which R(0) + ... +
 * R(i) > u_0 sum R (R = p where no mass is left, or no child was tested).
 * Children that come up when no mass is left (Z_k = 0, or at most 2^-24 of q)
 * are rejected.
 *
 * Tests are done in 64-bit floating point, sums in integers of 2^-46, so the
 * result does not depend on the order of the sums.
 *
 *  target, draft  device, [num_rows, vocab], DSPARK_PROB_FP32 or _BF16, row r at
 *                 r * stride elements; negative entries and NaN count as 0,
 *                 those above 1 as 1.  Any alignment (16-byte rows are read
 *                 faster).
 *  tokens         device, int64 [num_rows] (row 0's is not read).
 *  parents        device, int32 [num_rows], relative to the request's row 0.
 *  uniforms       device, fp32 [num_rows], in [0, 1): row i's decides its test,
 *                 row 0's the last token.  Below 0 and NaN count as 0.
 *  max_accepted   >= 1, at most 1023.
 *  out_tokens     device, int64 [num_requests, max_accepted + 1]: the accepted
 *                 tokens, the last token, then -1.
 *  out_rows       device, int32 [num_requests, max_accepted]: the accepted
 *                 tokens' rows, then -1 (what dspark_kv_compact takes).
 *  counts         device, int32 [num_requests]: accepted tokens.
 * A request without rows gets -1 and 0; one of more than 1024 rows too
 * (DSPARK_FLAG_LENGTH).  A drafted token outside [0, vocab) is rejected, one
 * whose parent is not a row before it is not tested (DSPARK_FLAG_ROW); a last row
 * without any probability gives token -1 (DSPARK_FLAG_ROW).  Outputs that overlap
 * one another or an input are refused.  A row's entries sum to less than 65,536 (they are probabilities).
 */
typedef enum { DSPARK_PROB_FP32 = 0, DSPARK_PROB_BF16 = 1 } dspark_prob_dtype;

int dspark_verify_drafts(const void *target, int target_dtype, int64_t target_stride, const void *draft,
                         int draft_dtype, int64_t draft_stride, int64_t num_rows, int64_t vocab,
                         const int64_t *tokens, const int32_t *parents, const float *uniforms,
                         const int32_t *row_start, int num_requests, int max_accepted, int replacement,
                         int64_t *out_tokens, int32_t *out_rows, int32_t *counts, unsigned int *error_flags,
                         cudaStream_t stream);

/*
 * dspark_kv_compact -- moves the accepted tokens' K|V together, in every
 * layer: of request b, the token at place context_lens[b] + rows[b][j] moves to
 * place context_lens[b] + first + j, for j < counts[b].
 *
 *  kv_caches      HOST, num_layers (1 to 1024) device pointers, no two alike;
 *                 block_scales: HOST, num_layers device pointers or NULL
 *                 (page-scaled caches).  Read before the call returns.
 *  rows           device, int32, row b at b * rows_stride, `width` entries:
 *                 ascending, rows[b][j] >= first + j.
 *  first          >= 0: 1 where row 0 is a token that stays.
 *  new_lens       device, int32 [num_requests], or NULL: receives
 *                 context_lens[b] + first + counts[b]; must not overlap
 *                 context_lens, rows or counts.
 * A request that had no rows in the step (a count of 0) grows by `first` like the others;
 * whoever keeps such a request in the batch keeps its old length too.
 * Requests must not share the pages that rows move into.  In a page-scaled cache
 * such a page's scale grows to the largest scale that comes in, and what it
 * holds is encoded anew.  A request whose counts, rows or places are out of range
 * is left out (DSPARK_FLAG_LENGTH), its new length its old one; a row in a page
 * out of range does not move (DSPARK_FLAG_BLOCK_RANGE).
 */
int dspark_kv_compact(void *const *kv_caches, int8_t *const *block_scales, int num_layers, int64_t num_blocks,
                      int num_kv_heads, int block_size, int head_dim, int kv_dtype, const int32_t *block_table,
                      int64_t table_stride, int64_t table_blocks, const int32_t *context_lens, int num_requests,
                      const int32_t *rows, int64_t rows_stride, int width, const int32_t *counts, int first,
                      int32_t *new_lens, unsigned int *error_flags, cudaStream_t stream);

/*
 * The page pool.  refs[page] is the number of block table entries that hold the
 * page; one with refs 0 is free.  pages[r] is the number of entries that row r of
 * the block table holds.  Pages are given out lowest number first, so what a
 * call gives out does not depend on timing.
 *
 * dspark_kv_fork -- pair i makes table row dst[i] a copy of row src[i]: the pages
 * full of its lens[src] tokens are shared (refs + 1), a last page that is not full
 * is copied into a free one in every layer, and dst has the same length.  Pages
 * that src holds beyond its tokens stay its own.  Row dst[i] must hold no
 * pages.
 *  src, dst       device, int32 [num_pairs], num_pairs <= 4096.  A pair whose
 *                 rows are out of range, whose dst holds pages, is a src of the
 *                 call or the dst of an earlier pair, or whose src's length does
 *                 not fit its pages, is left out (DSPARK_FLAG_LENGTH).  A pair
 *                 whose last page is out of range is left out, other entries out
 *                 of range are copied as they are (DSPARK_FLAG_BLOCK_RANGE).
 *                 The pairs that need a page get them in their order; those for
 *                 which there is none are left out (DSPARK_FLAG_PAGES).
 *  block_table, pages, lens, refs   device, int32, updated.
 *  workspace      device, 16-byte aligned, dspark_kv_fork_workspace bytes.
 *
 * dspark_kv_resize -- gives row r of the table the pages of tokens[r] tokens:
 * entries beyond them are given back (and set to -1), then missing ones are
 * taken, in the order of the rows.  0 tokens frees the row.  A row is served
 * where the pages asked for by it and all rows before it are there; others keep
 * what they hold (DSPARK_FLAG_PAGES).  A row whose tokens or pages do not fit the
 * table keeps its pages (DSPARK_FLAG_LENGTH).  An entry out of range is set to -1
 * (DSPARK_FLAG_BLOCK_RANGE), a page that nobody held stays free (DSPARK_FLAG_REFS).
 *  tokens         device, int32 [num_rows].
 *  workspace      device, 16-byte aligned, dspark_kv_resize_workspace bytes.
 */
int dspark_kv_fork(void *const *kv_caches, int8_t *const *block_scales, int num_layers, int64_t num_blocks,
                   int num_kv_heads, int block_size, int head_dim, int kv_dtype, int32_t *block_table,
                   int64_t table_stride, int64_t table_blocks, int32_t *pages, int32_t *lens, int num_rows,
                   const int32_t *src, const int32_t *dst, int num_pairs, int32_t *refs, void *workspace,
                   int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream);
int64_t dspark_kv_fork_workspace(int num_pairs);

int dspark_kv_resize(int32_t *block_table, int64_t table_stride, int64_t table_blocks, int32_t *pages,
                     const int32_t *tokens, int num_rows, int32_t *refs, int64_t num_blocks, int block_size,
                     void *workspace, int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream);
int64_t dspark_kv_resize_workspace(int num_rows, int64_t num_blocks);

/*
 * dspark_kv_insert_scaled -- stores new tokens' K and V in a page-scaled cache:
 * rows [query_start[b], query_start[b + 1]) go to the places behind request b's
 * context_lens[b] tokens.  A page's scale is the least e with |x| <= 448 * 2^e for
 * every finite new x of that page and head (K and V apart), and not below the
 * scale of a page that already holds some of the context's tokens, whose codes
 * are encoded anew where it grows.  Codes are e4m3(x * 2^-e), to nearest even;
 * infinities (and what exceeds 448 * 2^31) become the largest code, NaN stays.
 *
 *  k, v           device, bf16, element [t, h, d] at t * token_stride + h *
 *                 head_stride + d; 16-byte aligned, strides multiples of 8.
 * Pages that tokens go into belong to one request.  A request that does not fit
 * its table row is left out (DSPARK_FLAG_LENGTH), tokens of a page out of range
 * too (DSPARK_FLAG_BLOCK_RANGE).
 */
int dspark_kv_insert_scaled(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                            int64_t v_token_stride, int64_t v_head_stride, int64_t num_rows, void *kv_cache,
                            int8_t *block_scales, int64_t num_blocks, int num_kv_heads, int block_size, int head_dim,
                            const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                            const int32_t *query_start, const int32_t *context_lens, int num_requests,
                            unsigned int *error_flags, cudaStream_t stream);

/*
 * dspark_tree_attention_scaled -- dspark_tree_attention over a page-scaled cache
 * (kv_cache: e4m3 codes; block_scales in the place of k_scale and v_scale).  The
 * products take codes, exact in fp16; the scale of K multiplies the scores, that
 * of V the weights before they are rounded to fp16: 2^(s + e) for a token of V
 * scale e is off by at most 2^-11 of itself down to 2^-22 of the row's largest of
 * these, by 2^-33 of that below.  The other operators that read a cache
 * (dspark_attention_weight_accumulate, dspark_kv_evict, the writes) take its
 * per-tensor form only.
 */
int dspark_tree_attention_scaled(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_rows,
                                 int num_heads, int num_kv_heads, int head_dim, const void *kv_cache,
                                 const int8_t *block_scales, int64_t num_blocks, int block_size,
                                 const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                                 const int32_t *query_start, const int32_t *context_lens, int num_requests,
                                 int mask_kind, const uint64_t *tree_mask, int mask_words, float scale, void *out,
                                 float *lse, void *workspace, int64_t workspace_bytes, unsigned int *error_flags,
                                 cudaStream_t stream);
int64_t dspark_tree_attention_scaled_workspace(int64_t num_rows, int num_heads, int num_kv_heads, int head_dim,
                                               int num_requests);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_DRAFT_STEP_H */
