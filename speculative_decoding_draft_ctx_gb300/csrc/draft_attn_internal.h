// Internal interface between the host layer of the draft-attention operators
// (draft_attn_api.cpp) and their sm_103a kernels.  Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <cuda_runtime_api.h>

namespace dspark {

constexpr unsigned kFlagBlockRange = 0x10u;
constexpr unsigned kFlagLength = 0x20u;

constexpr int kScaleMin = -32, kScaleMax = 31;  // exponents of page-scaled caches

// ---------------------------------------------------------------- rope.cu

constexpr int kMaxRotary = 512;

struct RopeTableParams {
    void *out;
    int64_t first, count;
    int32_t rotary_dim;
    float amplitude;
    uint64_t turns[kMaxRotary / 2];  // frequency in turns per position, times 2^64
};

cudaError_t launch_rope_table(const RopeTableParams &p, bool fp32, cudaStream_t stream);

struct RopeInsertParams {
    const uint16_t *q, *k, *v;    // bf16 bits
    uint16_t *q_out, *k_out;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;  // elements
    const void *cos_sin;
    const int64_t *positions;
    const int64_t *slot_mapping;  // null: no insert
    unsigned char *cache;
    const float *k_scale, *v_scale;  // fp8 cache: device scalars (null = 1)
    unsigned int *error_flags;
    int64_t num_tokens, max_pos, capacity;
    int32_t num_heads, num_kv_heads, rotary_dim, block_size;
    bool interleaved, inverse, table_fp32, fp8;
    bool vec;  // every row 16-byte aligned and whole 8-element words rotate together
};

cudaError_t launch_rope_insert(const RopeInsertParams &p, int head_dim, cudaStream_t stream);

// ---------------------------------------------------------------- tree_attn*.cu

// What the attention and the weight accumulation read in common.
struct AttnParams {
    const uint16_t *q;  // bf16 bits
    int64_t q_ts, q_hs; // elements
    int64_t num_rows;
    const unsigned char *cache;
    const float *k_scale, *v_scale;
    const int8_t *block_scales;  // page-scaled caches: exponents [num_blocks, nkv, 2]; null otherwise
    const int32_t *table;
    int64_t table_stride, table_blocks;
    const int32_t *query_start, *context_lens;
    const uint64_t *tree_mask;
    unsigned int *error_flags;
    float *lse;         // attention: written; weight: read
    int64_t num_blocks;
    int32_t num_heads, num_kv_heads, group;  // group = num_heads / num_kv_heads
    int32_t block_size, num_requests;
    uint64_t block_magic;  // floor(2^64 / block_size) + 1; 0 for size 1
    int32_t mask_kind, mask_words;
    float scale;        // softmax scale
    uint64_t wait_ns;   // limit of every wait of the tensor-core kernels
    bool test_hold;     // test hook (see dspark::test_hold_ns): their producers copy nothing
    // attention
    uint16_t *out;
    float *parts;       // workspace: partial results, see tree_attn_mma.cuh
    // weight
    float *weights;
    int64_t weight_stride;
    float decay;
};

int64_t tree_attention_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, bool fp8,
                                 cudaError_t &e);
cudaError_t launch_tree_attention(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream);
// the same over a page-scaled cache (p.block_scales); the workspace covers both
int64_t tree_attention_scaled_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, cudaError_t &e);
cudaError_t launch_tree_attention_scaled(const AttnParams &p, int head_dim, cudaStream_t stream);
cudaError_t launch_attention_weight(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream);

// ---------------------------------------------------------------- kv_evict.cu

struct EvictParams {
    unsigned char *cache;
    const int32_t *table;
    int64_t table_stride, table_blocks;
    const int32_t *context_lens, *seq_lens;
    const float *weights;
    const int32_t *positions;
    float *weights_out;
    int32_t *positions_out, *new_lens;
    int32_t *counts;   // workspace: [B * H] moves, then
    int32_t *lists;    // [B * H][2][list_len]: places, then cache rows, given up and moved from
    unsigned int *error_flags;
    int64_t num_blocks, stride, list_len;
    int64_t budget, sinks, recent;
    int32_t num_requests, num_kv_heads, block_size;
    int32_t row_bytes;  // one token's K|V of one head
};

cudaError_t launch_kv_evict(const EvictParams &p, cudaStream_t stream);

}  // namespace dspark
