// Internal interface between the host layer of the draft-step operators
// (draft_step_api.cpp) and their sm_103a kernels.  Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <cuda_runtime_api.h>

#include "draft_attn_internal.h"

namespace dspark {

constexpr unsigned kFlagPages = 0x40u;
constexpr unsigned kFlagRow = 0x80u;
constexpr unsigned kFlagRefs = 0x100u;

// ---------------------------------------------------------------- verify.cu

constexpr int kVerifyRows = 1024;  // of one request

struct VerifyParams {
    const void *target, *draft;  // draft null: tokens taken without drawing
    int64_t target_stride, draft_stride, num_rows, vocab;
    const int64_t *tokens;
    const int32_t *parents;      // null: a chain
    const float *uniforms;
    const int32_t *row_start;
    int64_t *out_tokens;
    int32_t *out_rows, *counts;
    unsigned int *error_flags;
    int32_t num_requests, max_accepted;
    bool target_bf16, draft_bf16, replacement;
};

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream);

// ---------------------------------------------------------------- kv_pages.cu

constexpr int kMaxLayers = 64;  // of one launch: their addresses are kernel arguments
constexpr int kMaxPairs = 4096;

struct Layers {
    unsigned char *cache[kMaxLayers];
    int8_t *scales[kMaxLayers];  // [num_blocks, nkv, 2], or null
};

struct CompactParams {
    Layers layers;
    const int32_t *table;
    int64_t table_stride, table_blocks, num_blocks, rows_stride;
    const int32_t *context_lens, *rows, *counts;
    int32_t *new_lens;           // null: not written (or by an earlier launch)
    unsigned int *error_flags;
    int32_t num_layers, num_requests, num_kv_heads, block_size, row_bytes, width, first;
};

cudaError_t launch_compact(const CompactParams &p, bool scaled, cudaStream_t stream);

struct ForkParams {
    int32_t *table;
    int64_t table_stride, table_blocks, num_blocks;
    int32_t *pages, *lens, *refs;
    const int32_t *src, *dst;
    int4 *copies;                // workspace: per pair old page, new page, tokens to copy (0: none), whether it is done
    int32_t *free_list;          // workspace [num_pairs]
    unsigned int *error_flags;
    int32_t num_rows, num_pairs, block_size;
};

// the pages of the pairs' copies, of up to kMaxLayers layers
struct PageCopyParams {
    Layers layers;
    const int4 *copies;
    int32_t num_pairs, num_layers, num_kv_heads, block_size, row_bytes;
    bool scaled;
};

cudaError_t launch_fork(const ForkParams &p, cudaStream_t stream);
cudaError_t launch_page_copies(const PageCopyParams &p, cudaStream_t stream);

struct ResizeParams {
    int32_t *table;
    int64_t table_stride, table_blocks, num_blocks;
    int32_t *pages, *refs;
    const int32_t *tokens;
    int32_t *before;             // workspace [num_rows + 1]: pages asked for by the rows before
    int32_t *free_list;          // workspace [num_blocks]
    unsigned int *error_flags;
    int32_t num_rows, block_size;
};

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t stream);

// ---------------------------------------------------------------- kv_insert_scaled.cu

struct InsertScaledParams {
    const uint16_t *k, *v;  // bf16 bits
    int64_t k_ts, k_hs, v_ts, v_hs, num_rows;
    unsigned char *cache;
    int8_t *scales;
    const int32_t *table;
    int64_t table_stride, table_blocks, num_blocks;
    const int32_t *query_start, *context_lens;
    unsigned int *error_flags;
    int32_t num_requests, num_kv_heads, block_size, head_dim;
};

cudaError_t launch_insert_scaled(const InsertScaledParams &p, cudaStream_t stream);

}  // namespace dspark
