// What the host layers of the operators on the caches (draft_attn_api.cpp,
// draft_step_api.cpp) check alike.
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime_api.h>

#include "../../include/dspark_draft_attn.h"
#include "ctx_kv_internal.h"

namespace dspark {

inline int fail(int status, const char *fmt, ...)
{
    char text[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return api_fail(status, text);
}

inline int ok() { return api_fail(DSPARK_OK, ""); }

inline int launched(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? ok() : fail(DSPARK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The cache of every operator here; `rows` receives num_blocks * nkv * block_size.
inline int check_cache(const void *cache, int64_t num_blocks, int nkv, int block_size, int head_dim, int kv_dtype)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(DSPARK_ERR_INVALID_ARG, "head_dim %d not in {64, 128, 256}", head_dim);
    if (nkv < 1 || nkv > 65535)
        return fail(DSPARK_ERR_INVALID_ARG, "num_kv_heads %d not in [1, 65535]", nkv);
    if (block_size < 1)
        return fail(DSPARK_ERR_BLOCK_SIZE, "block size %d must be >= 1", block_size);
    if (kv_dtype != DSPARK_KV_BF16 && kv_dtype != DSPARK_KV_FP8_E4M3)
        return fail(DSPARK_ERR_DTYPE, "kv dtype %d unknown", kv_dtype);
    if (num_blocks < 1 || num_blocks > ((INT64_MAX / nkv) / block_size) / (4 * head_dim))
        return fail(DSPARK_ERR_INVALID_ARG, "cache of %lld blocks invalid", (long long)num_blocks);
    if (num_blocks * nkv * block_size >= (int64_t)UINT32_MAX)  // more rows than 32 bits number: beyond any device's memory
        return fail(DSPARK_ERR_INVALID_ARG, "cache of %lld blocks invalid", (long long)num_blocks);
    if (!cache)
        return fail(DSPARK_ERR_INVALID_ARG, "null kv_cache");
    if (!aligned(cache, 16))
        return fail(DSPARK_ERR_ALIGNMENT, "kv_cache must be 16-byte aligned");
    return DSPARK_OK;
}

// Places of a request: block table columns that lengths may reach (lengths
// are 32 bits; a tile past the last one must not overflow them).
inline int64_t usable_blocks(int64_t table_blocks, int block_size)
{
    return std::min<int64_t>(table_blocks, ((int64_t)INT32_MAX - 1024) / block_size);
}

inline int check_table(const int32_t *table, int64_t stride, int64_t blocks, int requests, const int32_t *lens)
{
    if (requests < 0 || requests > (1 << 24))
        return fail(DSPARK_ERR_INVALID_ARG, "num_requests %d not in [0, 2^24]", requests);
    if (blocks < 1 || stride < blocks || stride > (int64_t)1 << 40)
        return fail(DSPARK_ERR_INVALID_ARG, "block table of %lld entries a row, stride %lld", (long long)blocks,
                    (long long)stride);
    if (requests > 0 && (!table || !lens))
        return fail(DSPARK_ERR_INVALID_ARG, "null block_table or context_lens");
    if (!aligned(table, 4) || !aligned(lens, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "block_table and context_lens must be 4-byte aligned");
    return DSPARK_OK;
}

// Two arrays of n 4-byte entries that share some memory without being the same.
inline bool overlap_partly(const void *a, const void *b, int64_t n)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x != y && (x < y ? y - x : x - y) < (uint64_t)n * 4;
}

inline bool stride_ok(int64_t s) { return s >= -((int64_t)1 << 40) && s <= (int64_t)1 << 40; }

}  // namespace dspark
