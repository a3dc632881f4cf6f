/*
 * dspark_draft_attn.h -- C ABI of the operators that work on the paged caches
 * the context-KV write fills: the cos|sin table, rotary positions with the
 * K/V insert, the drafted tokens' attention, the attention weight the cached
 * tokens received, and the eviction by that weight.
 *
 * Every layer cache is [num_blocks, nkv, block_size, 2 * head_dim], K at
 * [0, head_dim), V at [head_dim, 2 * head_dim), bf16 or e4m3 codes, as
 * dspark_ctx_kv.h describes it; head_dim 64, 128 or 256, any block size >= 1.
 * A request's tokens are addressed through its row of a block table: its
 * token j sits in block table[b][j / block_size] at offset j % block_size.
 *
 * The conventions of dspark_ctx_kv.h hold: the caller owns every buffer, the
 * functions allocate, synchronise and copy nothing (all may be captured into
 * a CUDA graph), return a dspark_status and never throw.  Lengths, offsets
 * and block numbers live in device memory, so the kernels check them: what
 * is out of range is never dereferenced and raises a bit in *error_flags.
 * The waits inside the attention and the weight accumulation for their own
 * copies and products are bounded (4 s); one that ran out raises
 * DSPARK_FLAG_TIMEOUT, and that call's outputs hold nothing of use.  Their
 * allocation of tensor memory has no limit of its own: it waits for another
 * kernel's CTA on the same SM to free what it holds.
 */
#ifndef DSPARK_DRAFT_ATTN_H
#define DSPARK_DRAFT_ATTN_H

#include "dspark_ctx_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSPARK_FLAG_BLOCK_RANGE 0x10u /* a block table entry outside [0, num_blocks): its tokens are left out */
#define DSPARK_FLAG_LENGTH 0x20u      /* a length or offset outside its bounds: the request is left out */

/* How the drafted tokens of a request see one another. */
typedef enum {
    DSPARK_MASK_DENSE = 0,  /* every drafted token sees every other */
    DSPARK_MASK_CAUSAL = 1, /* itself and those before it */
    DSPARK_MASK_TREE = 2,   /* by a bit mask */
} dspark_draft_mask;

/*
 * dspark_rope_table -- the cos|sin table the write, the inserts and
 * dspark_rope_kv_insert read:
 *   out[p, i]       = amplitude * cos((first_position + p) * freqs[i])
 *   out[p, r/2 + i] = amplitude * sin((first_position + p) * freqs[i]).
 *
 *  out        device, [num_positions, rotary_dim], bf16 (out_fp32 0) or fp32
 *             (1), 16-byte aligned.
 *  freqs      HOST, double [rotary_dim / 2], radians per position, finite;
 *             read before the call returns.
 *  rotary_dim even, 2..512;  0 <= first_position,
 *             first_position + num_positions <= 2^31.
 * The angle is reduced exactly (a 64-bit fixed-point fraction of a turn), so
 * far positions lose nothing beyond the frequency's own rounding.
 */
int dspark_rope_table(void *out, int64_t first_position, int64_t num_positions, int rotary_dim, const double *freqs,
                      double amplitude, int out_fp32, cudaStream_t stream);

/*
 * dspark_rope_kv_insert -- rotary positions of drafted (or context) tokens
 * that take no QK norm, with their optional K/V insert.  One launch.
 *
 *  q, k, v       device, bf16, element [t, h, d] at t * token_stride +
 *                h * head_stride + d (strides in elements): views of a packed
 *                qkv, for instance.  v is read only by calls that insert
 *                (NULL otherwise).  2-byte aligned; 16-byte rows take wider
 *                loads.
 *  q_out, k_out  device, bf16, with strides of their own; may be q and k
 *                themselves (same strides: in place), must not overlap them
 *                otherwise.
 *  cos_sin       device, [max_pos, rotary_dim], bf16 or fp32
 *                (cos_sin_fp32), 16-byte aligned, cos in [0, r/2), sin in
 *                [r/2, r).
 *  positions     device, int64 [num_tokens].  A token whose position lies
 *                outside the table comes out unrotated, is not inserted and
 *                raises DSPARK_FLAG_POS_RANGE.
 *  head_dim      64, 128 or 256;  rotary_dim even, 2..head_dim: the leading
 *                dims that turn; the others pass.
 *  interleaved   0: dim i pairs with i + r/2; 1: dim 2i with 2i + 1.
 *                (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), fp32, rounded once.
 *  inverse       1: the transposed rotation (s negated): the gradient of the
 *                rotation with respect to its input.
 *  slot_mapping, kv_cache, num_blocks, block_size, kv_dtype, k_scale,
 *  v_scale       the insert, both pointers or neither: tokens with slot >= 0
 *                have K' (as rounded to bf16) and V stored, bf16 or e4m3 of
 *                x / scale (device scalars, NULL means 1).  Valid slots must
 *                be distinct; one beyond the cache is not inserted and raises
 *                DSPARK_FLAG_SLOT_RANGE.
 * num_tokens == 0 returns DSPARK_OK without a launch.
 */
int dspark_rope_kv_insert(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                          int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                          int64_t v_head_stride, void *q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                          void *k_out, int64_t ko_token_stride, int64_t ko_head_stride, const void *cos_sin,
                          int cos_sin_fp32, int64_t max_pos, const int64_t *positions, int64_t num_tokens,
                          int num_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int inverse,
                          const int64_t *slot_mapping, void *kv_cache, int64_t num_blocks, int block_size,
                          int kv_dtype, const float *k_scale, const float *v_scale, unsigned int *error_flags,
                          cudaStream_t stream);

/*
 * dspark_tree_attention -- the drafted tokens' attention over the paged
 * cache.  Request b has context_lens[b] context tokens at places
 * [0, context_lens[b]) of its block table row, then its drafted tokens'
 * K/V at the places that follow (inserted before this call).  Drafted token
 * i (row t = query_start[b] + i of q) sees every context token and the
 * drafted tokens that the mask gives it:
 *   out[t, h]  = sum_j softmax_j(scale * q[t, h] . k_j) v_j
 *   lse[t, h]  = log sum_j exp(scale * q[t, h] . k_j)     (natural log)
 * with KV head h / (num_heads / num_kv_heads).  Scores, statistics and sums are
 * fp32.  For the product with V the weights are rounded to 16 bits: to bf16
 * over a bf16 cache (each by at most 2^-8 of itself), to fp16 over an fp8 cache
 * (2^-11 down to 2^-28 of the row's largest weight, 2^-39 of the largest below,
 * where scores stay below 2^19, beyond which fp32 tells them apart by 1/16 at
 * best; the queries to fp16 too, by at most 2^-24 of their row's largest
 * element).
 * out is rounded to bf16 once.  A row that sees nothing gives zeros and -inf.  Tokens that a row does not see do not reach its result,
 * whatever their K and V hold (NaN and infinities included).
 *
 *  q             device, bf16, element [t, h, d] at t * token_stride +
 *                h * head_stride + d; 16-byte aligned, strides multiples of 8.
 *  kv_cache      device, 16-byte aligned; k_scale, v_scale: device fp32
 *                scalars of an fp8 cache (NULL means 1), ignored for bf16.
 *  block_table   device, int32, row b at b * table_stride, table_blocks
 *                entries each (those beyond a request's length are not read).
 *  query_start   device, int32 [num_requests + 1]: rows [query_start[b],
 *                query_start[b + 1]) of q are request b's; rows of no request
 *                are left as they were in out and lse.
 *  context_lens  device, int32 [num_requests].
 *  mask_kind     a dspark_draft_mask; tree_mask: device, [num_rows,
 *                mask_words] 64-bit words, bit j % 64 of word j / 64 of row t:
 *                the row sees its request's drafted token j (not read
 *                otherwise).  A request of more than 64 * mask_words drafted
 *                tokens is left out (DSPARK_FLAG_LENGTH).
 *  scale         finite.
 *  out           device, bf16 [num_rows, num_heads, head_dim], 16-byte
 *                aligned; lse: device, fp32 [num_rows, num_heads].
 *  workspace     device, 16-byte aligned, dspark_tree_attention_workspace
 *                bytes; needs no initial contents and holds nothing between
 *                calls.  Calls that can overlap on the GPU need one each.
 * num_rows == 0 or num_requests == 0 returns DSPARK_OK without a launch.
 */
int dspark_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_rows,
                          int num_heads, int num_kv_heads, int head_dim, const void *kv_cache, int64_t num_blocks,
                          int block_size, int kv_dtype, const float *k_scale, const float *v_scale,
                          const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                          const int32_t *query_start, const int32_t *context_lens, int num_requests, int mask_kind,
                          const uint64_t *tree_mask, int mask_words, float scale, void *out, float *lse,
                          void *workspace, int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream);

/* Bytes of workspace that dspark_tree_attention needs for these sizes on the
 * current device (0: none), or -1 with dspark_ctx_kv_last_error set. */
int64_t dspark_tree_attention_workspace(int64_t num_rows, int num_heads, int num_kv_heads, int head_dim,
                                        int num_requests, int kv_dtype);

/*
 * dspark_attention_weight_accumulate -- the attention weight each context
 * token received from the drafted tokens' queries, per KV head:
 *   weights[b, h, j] = decay * weights[b, h, j]
 *                    + sum_{i, g} exp(scale * q[t_i, h G + g] . k_j - lse[t_i, h G + g])
 * for j < context_lens[b], with lse as dspark_tree_attention wrote it (a row
 * whose lse is -inf saw nothing and adds nothing, whatever its query holds);
 * other entries stay.  A token
 * in a block out of range receives nothing: its weight only decays
 * (DSPARK_FLAG_BLOCK_RANGE where the request has drafted tokens).  The sums run
 * in a fixed order.
 *
 *  weights       device, fp32 [num_requests, num_kv_heads, weight_stride];
 *                a request of more than weight_stride context tokens is left
 *                out (DSPARK_FLAG_LENGTH).
 *  Other arguments as dspark_tree_attention.
 */
int dspark_attention_weight_accumulate(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_rows,
                                       int num_heads, int num_kv_heads, int head_dim, const void *kv_cache,
                                       int64_t num_blocks, int block_size, int kv_dtype, const float *k_scale,
                                       const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                                       const int32_t *query_start, const int32_t *context_lens, int num_requests,
                                       const float *lse, float scale, float decay, float *weights,
                                       int64_t weight_stride, unsigned int *error_flags, cudaStream_t stream);

/*
 * dspark_kv_evict -- keeps the `budget` heaviest context tokens of every
 * (request, KV head) and frees the rest.  Of a request with n =
 * context_lens[b] > budget tokens, each KV head keeps budget: first those
 * whose position is below `sinks` or at least seq_lens[b] - recent, then by
 * falling weight (NaN last), ties to the lowest place.  Kept tokens at places
 * >= budget move into the places below budget that were given up, the i-th
 * such token into the i-th such place, so no other token moves (softmax does
 * not depend on the order).  K|V rows move in the cache, weights and
 * positions with them; places [budget, n) then hold weight 0 and position -1.
 * A request with n <= budget is left as it is.
 *
 *  kv_cache      device, rows of 2 * head_dim elements, as above.  Requests
 *                must not share blocks.
 *  weights       device, fp32 [num_requests, num_kv_heads, stride];
 *  positions     device, int32, same shape: the sequence position of the
 *                token at each place.
 *  weights_out,  device, same shape: the results, places behind a request's
 *  positions_out length copied; may be weights and positions themselves (in
 *                place), must not overlap them otherwise.
 *  seq_lens      device, int32 [num_requests]: positions seen so far.
 *  new_lens      device, int32 [num_requests]: receives min(n, budget) (a
 *                request left out for a bad length: its n); may be context_lens
 *                or seq_lens itself (in place), must not overlap them otherwise.
 *  budget >= 1, sinks >= 0, recent >= 0, sinks + recent <= budget.
 *  workspace     device, 16-byte aligned, dspark_kv_evict_workspace bytes.
 * A request whose length exceeds stride or its table row is left out
 * (DSPARK_FLAG_LENGTH); a row in a block out of range does not move
 * (DSPARK_FLAG_BLOCK_RANGE).
 */
int dspark_kv_evict(void *kv_cache, int64_t num_blocks, int num_kv_heads, int block_size, int head_dim, int kv_dtype,
                    const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                    const int32_t *context_lens, int num_requests, const float *weights, const int32_t *positions,
                    float *weights_out, int32_t *positions_out, int64_t stride, const int32_t *seq_lens,
                    int64_t budget, int64_t sinks, int64_t recent, int32_t *new_lens, void *workspace,
                    int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream);

/* Bytes of workspace that dspark_kv_evict needs, or -1 with
 * dspark_ctx_kv_last_error set. */
int64_t dspark_kv_evict_workspace(int num_requests, int num_kv_heads, int64_t stride, int64_t budget);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_DRAFT_ATTN_H */
