// C-ABI host layer of the draft-step operators (dspark_draft_step.h): argument
// checks and launches.
#include "../../include/dspark_draft_step.h"

#include "ctx_kv_internal.h"
#include "draft_api_checks.h"
#include "draft_step_internal.h"

namespace {

using namespace dspark;

// The layers' caches and, in a page-scaled cache, their exponents.
int check_layers(void *const *caches, int8_t *const *scales, int num_layers, int64_t num_blocks, int nkv, int block_size,
                 int head_dim, int kv_dtype)
{
    if (num_layers < 1 || num_layers > 1024)
        return fail(DSPARK_ERR_INVALID_ARG, "num_layers %d not in [1, 1024]", num_layers);
    if (!caches)
        return fail(DSPARK_ERR_INVALID_ARG, "null kv_caches");
    const int st = check_cache(caches[0], num_blocks, nkv, block_size, head_dim, kv_dtype);
    if (st != DSPARK_OK)
        return st;
    if (scales && kv_dtype != DSPARK_KV_FP8_E4M3)
        return fail(DSPARK_ERR_DTYPE, "block_scales belong to caches of e4m3 codes");
    for (int l = 0; l < num_layers; l++) {
        if (!caches[l] || (scales && !scales[l]))
            return fail(DSPARK_ERR_INVALID_ARG, "null cache or block_scales of layer %d", l);
        if (!aligned(caches[l], 16))
            return fail(DSPARK_ERR_ALIGNMENT, "cache of layer %d must be 16-byte aligned", l);
        for (int k = 0; k < l; k++)
            if (caches[k] == caches[l] || (scales && scales[k] == scales[l]))
                return fail(DSPARK_ERR_INVALID_ARG, "layers %d and %d have the same cache or block_scales", k, l);
    }
    return DSPARK_OK;
}

void layers_from(Layers &to, void *const *caches, int8_t *const *scales, int first, int count)
{
    for (int l = 0; l < count; l++) {
        to.cache[l] = static_cast<unsigned char *>(caches[first + l]);
        to.scales[l] = scales ? scales[first + l] : nullptr;
    }
}

bool overlap(const void *a, int64_t an, const void *b, int64_t bn)  // of an and bn bytes
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uint64_t)bn && y < x + (uint64_t)an;
}

// Whether `bytes` bytes from `out` on share any with `rows` rows of `width` bytes, `stride` bytes apart (either way).
bool overlap_rows(const void *out, int64_t bytes, const void *at, int64_t rows, int64_t width, int64_t stride)
{
    if (bytes < 1 || rows < 1 || width < 1)
        return false;
    __int128 x = (__int128)reinterpret_cast<uintptr_t>(at) - (__int128)reinterpret_cast<uintptr_t>(out), s = stride;
    if (s < 0) {
        x += (rows - 1) * s;
        s = -s;
    }
    // row r is [x + r s, x + r s + width) there: the first that ends behind 0 begins before `bytes`
    const __int128 r = x + width > 0 ? 0 : s == 0 ? rows : -(x + width) / s + 1;
    return r < rows && x + r * s < bytes;
}

// Rows of the block table that a call changes.
int check_pool(const int32_t *table, int64_t stride, int64_t blocks, int rows, const int32_t *pages, const int32_t *refs,
               int64_t num_blocks, int block_size)
{
    const int st = check_table(table, stride, blocks, rows, pages);
    if (st != DSPARK_OK)
        return st;
    if (block_size < 1)
        return fail(DSPARK_ERR_BLOCK_SIZE, "block size %d must be >= 1", block_size);
    if (num_blocks < 1 || num_blocks >= INT32_MAX)
        return fail(DSPARK_ERR_INVALID_ARG, "pool of %lld pages invalid", (long long)num_blocks);
    if (rows > 0 && !refs)
        return fail(DSPARK_ERR_INVALID_ARG, "null refs");
    if (!aligned(refs, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "refs must be 4-byte aligned");
    return DSPARK_OK;
}

}  // namespace

extern "C" {

int dspark_verify_drafts(const void *target, int target_dtype, int64_t target_stride, const void *draft,
                         int draft_dtype, int64_t draft_stride, int64_t num_rows, int64_t vocab,
                         const int64_t *tokens, const int32_t *parents, const float *uniforms,
                         const int32_t *row_start, int num_requests, int max_accepted, int replacement,
                         int64_t *out_tokens, int32_t *out_rows, int32_t *counts, unsigned int *error_flags,
                         cudaStream_t stream)
{
    if ((target_dtype != DSPARK_PROB_FP32 && target_dtype != DSPARK_PROB_BF16) ||
        (draft && draft_dtype != DSPARK_PROB_FP32 && draft_dtype != DSPARK_PROB_BF16))
        return fail(DSPARK_ERR_DTYPE, "probability dtype %d or %d unknown", target_dtype, draft_dtype);
    if (vocab < 1 || vocab > (1 << 30))
        return fail(DSPARK_ERR_INVALID_ARG, "vocab %lld not in [1, 2^30]", (long long)vocab);
    if (num_rows < 0 || num_rows > INT32_MAX)
        return fail(DSPARK_ERR_INVALID_ARG, "num_rows %lld out of range", (long long)num_rows);
    if (num_requests < 0 || num_requests > (1 << 24))
        return fail(DSPARK_ERR_INVALID_ARG, "num_requests %d not in [0, 2^24]", num_requests);
    if (max_accepted < 1 || max_accepted >= kVerifyRows)
        return fail(DSPARK_ERR_INVALID_ARG, "max_accepted %d not in [1, %d]", max_accepted, kVerifyRows - 1);
    if (!stride_ok(target_stride) || (draft && !stride_ok(draft_stride)))
        return fail(DSPARK_ERR_INVALID_ARG, "row stride out of range");
    if (num_requests == 0)
        return ok();
    if (!row_start || !out_tokens || !out_rows || !counts)
        return fail(DSPARK_ERR_INVALID_ARG, "null row_start, out_tokens, out_rows or counts");
    if (num_rows > 0 && (!target || !tokens || !uniforms))
        return fail(DSPARK_ERR_INVALID_ARG, "null target, tokens or uniforms");
    if (!aligned(target, target_dtype == DSPARK_PROB_BF16 ? 2 : 4) || !aligned(draft, draft_dtype == DSPARK_PROB_BF16 ? 2 : 4) ||
        !aligned(tokens, 8) || !aligned(out_tokens, 8) || !aligned(parents, 4) || !aligned(uniforms, 4) ||
        !aligned(row_start, 4) || !aligned(out_rows, 4) || !aligned(counts, 4) || !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "buffers must be aligned to their element's size");
    const int64_t T = num_rows, B = num_requests, t_size = target_dtype == DSPARK_PROB_BF16 ? 2 : 4, d_size = draft_dtype == DSPARK_PROB_BF16 ? 2 : 4;
    const struct {
        const void *at;
        int64_t bytes;
    } used[] = {{out_tokens, B * (max_accepted + 1) * 8}, {out_rows, B * max_accepted * 4}, {counts, B * 4}, {row_start, (B + 1) * 4},
                {tokens, T * 8}, {uniforms, T * 4}, {parents, parents ? T * 4 : 0}};
    for (int i = 0; i < 3; i++) {
        bool shared = overlap_rows(used[i].at, used[i].bytes, target, T, vocab * t_size, target_stride * t_size) ||
                      overlap_rows(used[i].at, used[i].bytes, draft, draft ? T : 0, vocab * d_size, draft_stride * d_size);
        for (int k = i + 1; k < 7; k++)
            shared |= used[k].bytes > 0 && overlap(used[i].at, used[i].bytes, used[k].at, used[k].bytes);
        if (shared)
            return fail(DSPARK_ERR_INVALID_ARG, "out_tokens, out_rows or counts overlap one another or an input");
    }
    VerifyParams p{};
    p.target = target;
    p.draft = draft;
    p.target_stride = target_stride;
    p.draft_stride = draft_stride;
    p.num_rows = num_rows;
    p.vocab = vocab;
    p.tokens = tokens;
    p.parents = parents;
    p.uniforms = uniforms;
    p.row_start = row_start;
    p.out_tokens = out_tokens;
    p.out_rows = out_rows;
    p.counts = counts;
    p.error_flags = error_flags;
    p.num_requests = num_requests;
    p.max_accepted = max_accepted;
    p.target_bf16 = target_dtype == DSPARK_PROB_BF16;
    p.draft_bf16 = draft_dtype == DSPARK_PROB_BF16;
    p.replacement = replacement != 0;
    return launched(launch_verify(p, stream), "verify drafts");
}

int dspark_kv_compact(void *const *kv_caches, int8_t *const *block_scales, int num_layers, int64_t num_blocks,
                      int num_kv_heads, int block_size, int head_dim, int kv_dtype, const int32_t *block_table,
                      int64_t table_stride, int64_t table_blocks, const int32_t *context_lens, int num_requests,
                      const int32_t *rows, int64_t rows_stride, int width, const int32_t *counts, int first,
                      int32_t *new_lens, unsigned int *error_flags, cudaStream_t stream)
{
    int st = check_layers(kv_caches, block_scales, num_layers, num_blocks, num_kv_heads, block_size, head_dim, kv_dtype);
    if (st != DSPARK_OK || (st = check_table(block_table, table_stride, table_blocks, num_requests, context_lens)) != DSPARK_OK)
        return st;
    if (width < 0 || rows_stride < width || rows_stride > (int64_t)1 << 40)
        return fail(DSPARK_ERR_INVALID_ARG, "rows of %d entries, stride %lld", width, (long long)rows_stride);
    if (first < 0)
        return fail(DSPARK_ERR_INVALID_ARG, "first %d must be >= 0", first);
    if (num_requests == 0)
        return ok();
    if (!counts || (width > 0 && !rows))
        return fail(DSPARK_ERR_INVALID_ARG, "null rows or counts");
    if (!aligned(rows, 4) || !aligned(counts, 4) || !aligned(new_lens, 4) || !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "rows, counts, new_lens and error_flags must be 4-byte aligned");
    const int64_t bytes = (int64_t)num_requests * 4;
    if (new_lens && (overlap(new_lens, bytes, context_lens, bytes) || overlap(new_lens, bytes, counts, bytes) ||
                     (width > 0 && overlap(new_lens, bytes, rows, ((num_requests - 1) * rows_stride + width) * 4))))
        return fail(DSPARK_ERR_INVALID_ARG, "new_lens overlaps context_lens, rows or counts");
    CompactParams p{};
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.num_blocks = num_blocks;
    p.rows_stride = rows_stride;
    p.context_lens = context_lens;
    p.rows = rows;
    p.counts = counts;
    p.error_flags = error_flags;
    p.num_requests = num_requests;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.row_bytes = 2 * head_dim * (kv_dtype == DSPARK_KV_FP8_E4M3 ? 1 : 2);
    p.width = width;
    p.first = first;
    for (int l = 0; l < num_layers; l += kMaxLayers) {
        p.num_layers = num_layers - l < kMaxLayers ? num_layers - l : kMaxLayers;
        p.new_lens = l ? nullptr : new_lens;
        layers_from(p.layers, kv_caches, block_scales, l, p.num_layers);
        const cudaError_t e = launch_compact(p, block_scales != nullptr, stream);
        if (e != cudaSuccess)
            return launched(e, "compact");
    }
    return ok();
}

int64_t dspark_kv_fork_workspace(int num_pairs)
{
    if (num_pairs < 0 || num_pairs > kMaxPairs) {
        fail(DSPARK_ERR_INVALID_ARG, "%d pairs not in [0, %d]", num_pairs, kMaxPairs);
        return -1;
    }
    return (int64_t)num_pairs * 5 * 4;  // the copies and the free pages
}

int dspark_kv_fork(void *const *kv_caches, int8_t *const *block_scales, int num_layers, int64_t num_blocks,
                   int num_kv_heads, int block_size, int head_dim, int kv_dtype, int32_t *block_table,
                   int64_t table_stride, int64_t table_blocks, int32_t *pages, int32_t *lens, int num_rows,
                   const int32_t *src, const int32_t *dst, int num_pairs, int32_t *refs, void *workspace,
                   int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream)
{
    int st = check_layers(kv_caches, block_scales, num_layers, num_blocks, num_kv_heads, block_size, head_dim, kv_dtype);
    if (st != DSPARK_OK ||
        (st = check_pool(block_table, table_stride, table_blocks, num_rows, pages, refs, num_blocks, block_size)) != DSPARK_OK)
        return st;
    const int64_t need = dspark_kv_fork_workspace(num_pairs);
    if (need < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (num_pairs == 0 || num_rows == 0)
        return ok();
    if (!lens || !src || !dst)
        return fail(DSPARK_ERR_INVALID_ARG, "null lens, src or dst");
    if (!aligned(lens, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(error_flags, 4) || !aligned(workspace, 16))
        return fail(DSPARK_ERR_ALIGNMENT, "workspace must be 16-byte, the other buffers 4-byte aligned");
    if (workspace_bytes < need || !workspace)
        return fail(DSPARK_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
    const int64_t table_bytes = ((num_rows - 1) * table_stride + table_blocks) * 4;
    const struct {
        const void *at;
        int64_t bytes;
    } used[] = {{block_table, table_bytes}, {pages, (int64_t)num_rows * 4}, {lens, (int64_t)num_rows * 4}, {refs, num_blocks * 4},
                {src, (int64_t)num_pairs * 4}, {dst, (int64_t)num_pairs * 4}};
    for (int i = 0; i < 4; i++)
        for (int k = i + 1; k < 6; k++)
            if (overlap(used[i].at, used[i].bytes, used[k].at, used[k].bytes))
                return fail(DSPARK_ERR_INVALID_ARG, "block_table, pages, lens, refs, src or dst overlap");
    ForkParams p{};
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.num_blocks = num_blocks;
    p.pages = pages;
    p.lens = lens;
    p.refs = refs;
    p.src = src;
    p.dst = dst;
    p.copies = static_cast<int4 *>(workspace);
    p.free_list = reinterpret_cast<int32_t *>(p.copies + num_pairs);
    p.error_flags = error_flags;
    p.num_rows = num_rows;
    p.num_pairs = num_pairs;
    p.block_size = block_size;
    cudaError_t e = launch_fork(p, stream);
    PageCopyParams c{};
    c.copies = p.copies;
    c.num_pairs = num_pairs;
    c.num_kv_heads = num_kv_heads;
    c.block_size = block_size;
    c.row_bytes = 2 * head_dim * (kv_dtype == DSPARK_KV_FP8_E4M3 ? 1 : 2);
    c.scaled = block_scales != nullptr;
    for (int l = 0; l < num_layers && e == cudaSuccess && block_size > 1; l += kMaxLayers) {  // (pages of one token are never part full)
        c.num_layers = num_layers - l < kMaxLayers ? num_layers - l : kMaxLayers;
        layers_from(c.layers, kv_caches, block_scales, l, c.num_layers);
        e = launch_page_copies(c, stream);
    }
    return launched(e, "fork");
}

int64_t dspark_kv_resize_workspace(int num_rows, int64_t num_blocks)
{
    if (num_rows < 0 || num_rows > (1 << 24) || num_blocks < 1 || num_blocks >= INT32_MAX) {
        fail(DSPARK_ERR_INVALID_ARG, "%d rows not in [0, 2^24] or %lld pages not in [1, 2^31 - 1)", num_rows, (long long)num_blocks);
        return -1;
    }
    return num_rows ? ((int64_t)num_rows + 1 + num_blocks) * 4 : 0;  // what the rows ask for and the free pages
}

int dspark_kv_resize(int32_t *block_table, int64_t table_stride, int64_t table_blocks, int32_t *pages,
                     const int32_t *tokens, int num_rows, int32_t *refs, int64_t num_blocks, int block_size,
                     void *workspace, int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream)
{
    const int st = check_pool(block_table, table_stride, table_blocks, num_rows, pages, refs, num_blocks, block_size);
    if (st != DSPARK_OK)
        return st;
    if (num_rows == 0)
        return ok();
    if (!tokens)
        return fail(DSPARK_ERR_INVALID_ARG, "null tokens");
    if (!aligned(tokens, 4) || !aligned(error_flags, 4) || !aligned(workspace, 16))
        return fail(DSPARK_ERR_ALIGNMENT, "workspace must be 16-byte, the other buffers 4-byte aligned");
    const int64_t need = dspark_kv_resize_workspace(num_rows, num_blocks), rows_bytes = (int64_t)num_rows * 4;
    if (workspace_bytes < need || !workspace)
        return fail(DSPARK_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
    const int64_t table_bytes = ((num_rows - 1) * table_stride + table_blocks) * 4;
    if (overlap(block_table, table_bytes, pages, rows_bytes) || overlap(block_table, table_bytes, tokens, rows_bytes) ||
        overlap(block_table, table_bytes, refs, num_blocks * 4) || overlap(pages, rows_bytes, tokens, rows_bytes) ||
        overlap(pages, rows_bytes, refs, num_blocks * 4) || overlap(tokens, rows_bytes, refs, num_blocks * 4))
        return fail(DSPARK_ERR_INVALID_ARG, "block_table, pages, tokens or refs overlap");
    ResizeParams p{};
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.num_blocks = num_blocks;
    p.pages = pages;
    p.refs = refs;
    p.tokens = tokens;
    p.before = static_cast<int32_t *>(workspace);
    p.free_list = p.before + num_rows + 1;
    p.error_flags = error_flags;
    p.num_rows = num_rows;
    p.block_size = block_size;
    return launched(launch_resize(p, stream), "resize");
}

int dspark_kv_insert_scaled(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                            int64_t v_token_stride, int64_t v_head_stride, int64_t num_rows, void *kv_cache,
                            int8_t *block_scales, int64_t num_blocks, int num_kv_heads, int block_size, int head_dim,
                            const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                            const int32_t *query_start, const int32_t *context_lens, int num_requests,
                            unsigned int *error_flags, cudaStream_t stream)
{
    int st = check_cache(kv_cache, num_blocks, num_kv_heads, block_size, head_dim, DSPARK_KV_FP8_E4M3);
    if (st != DSPARK_OK || (st = check_table(block_table, table_stride, table_blocks, num_requests, context_lens)) != DSPARK_OK)
        return st;
    if (num_rows < 0 || num_rows > INT32_MAX)
        return fail(DSPARK_ERR_INVALID_ARG, "num_rows %lld out of range", (long long)num_rows);
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (!stride_ok(s) || s % 8 != 0)
            return fail(DSPARK_ERR_ALIGNMENT, "strides of k and v must be multiples of 8 elements");
    if (num_rows == 0 || num_requests == 0)
        return ok();
    if (!k || !v || !block_scales || !query_start)
        return fail(DSPARK_ERR_INVALID_ARG, "null k, v, block_scales or query_start");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(query_start, 4) || !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "k and v must be 16-byte, query_start and error_flags 4-byte aligned");
    InsertScaledParams p{};
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_ts = k_token_stride, p.k_hs = k_head_stride;
    p.v_ts = v_token_stride, p.v_hs = v_head_stride;
    p.num_rows = num_rows;
    p.cache = static_cast<unsigned char *>(kv_cache);
    p.scales = block_scales;
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.num_blocks = num_blocks;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.error_flags = error_flags;
    p.num_requests = num_requests;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.head_dim = head_dim;
    return launched(launch_insert_scaled(p, stream), "scaled insert");
}

}  // extern "C"
