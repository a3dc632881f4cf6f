// C-ABI host layer of the draft-attention operators (dspark_draft_attn.h):
// argument checks and launches.
#include "../../include/dspark_draft_attn.h"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace {

using namespace dspark;

constexpr uint64_t kWaitNs = 4000000000;  // of a wait inside a kernel, which takes microseconds

int fail(int status, const char *fmt, ...)
{
    char text[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return api_fail(status, text);
}

int ok() { return api_fail(DSPARK_OK, ""); }

int launched(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? ok() : fail(DSPARK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The cache of every operator here; `rows` receives num_blocks * nkv * block_size.
int check_cache(const void *cache, int64_t num_blocks, int nkv, int block_size, int head_dim, int kv_dtype)
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
int64_t usable_blocks(int64_t table_blocks, int block_size)
{
    return std::min<int64_t>(table_blocks, ((int64_t)INT32_MAX - 1024) / block_size);
}

int check_table(const int32_t *table, int64_t stride, int64_t blocks, int requests, const int32_t *lens)
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
bool overlap_partly(const void *a, const void *b, int64_t n)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x != y && (x < y ? y - x : x - y) < (uint64_t)n * 4;
}

// f radians as a fraction of a turn in units of 2^-64, off by one at most:
// whole turns do not matter (positions are whole).  The quotient by 2 pi (its
// first 107 bits) is taken as a double and what that leaves over; a double
// alone is off by 2^-56 of a turn for f near 1, 2^-22 radians at position 2^31.
uint64_t fraction_of_a_turn(double f)
{
    constexpr double kTwoPi = 6.283185307179586232, kTwoPiRest = 2.4492935982947064e-16;
    const double q = f / kTwoPi;
    const double rest = (std::fma(-q, kTwoPi, f) - q * kTwoPiRest) / kTwoPi;
    const double a = std::nearbyint(std::ldexp(q - std::floor(q), 64));       // in [0, 2^64]
    const double b = std::nearbyint(std::ldexp(rest - std::nearbyint(rest), 64));  // in [-2^63, 2^63]
    const uint64_t whole = a >= 18446744073709551616.0 ? 0u : (uint64_t)a;
    return b >= 0.0 ? whole + (uint64_t)b : whole - (uint64_t)-b;
}

bool stride_ok(int64_t s) { return s >= -((int64_t)1 << 40) && s <= (int64_t)1 << 40; }

// The sizes that the calls and their workspace queries refuse alike.
bool attention_sizes_ok(int64_t rows, int heads, int nkv, int requests)
{
    return nkv >= 1 && nkv <= 65535 && heads >= 1 && heads % nkv == 0 && heads <= (1 << 20) && rows >= 0 &&
           rows <= ((int64_t)INT32_MAX - 1024) / (heads / nkv) && requests >= 0 && requests <= (1 << 24);
}
bool evict_sizes_ok(int requests, int nkv, int64_t stride)
{
    return requests >= 0 && nkv >= 1 && (int64_t)requests * nkv <= ((int64_t)1 << 31) / 16 - 1 && stride >= 0 &&
           stride <= (int64_t)INT32_MAX - 1024;
}

// What the attention and the weight accumulation check alike.
int check_attention(AttnParams &p, const void *q, int64_t q_ts, int64_t q_hs, int64_t rows, int heads, int nkv,
                    int head_dim, const void *cache, int64_t num_blocks, int block_size, int kv_dtype,
                    const float *k_scale, const float *v_scale, const int32_t *table, int64_t table_stride,
                    int64_t table_blocks, const int32_t *query_start, const int32_t *lens, int requests, float scale,
                    unsigned int *error_flags)
{
    int st = check_cache(cache, num_blocks, nkv, block_size, head_dim, kv_dtype);
    if (st != DSPARK_OK)
        return st;
    if ((st = check_table(table, table_stride, table_blocks, requests, lens)) != DSPARK_OK)
        return st;
    if (heads < 1 || heads % nkv != 0 || heads > (1 << 20))
        return fail(DSPARK_ERR_INVALID_ARG, "num_heads %d is not a multiple of num_kv_heads %d", heads, nkv);
    if (rows < 0 || rows > ((int64_t)INT32_MAX - 1024) / (heads / nkv))
        return fail(DSPARK_ERR_INVALID_ARG, "num_rows %lld out of range", (long long)rows);
    if (!std::isfinite(scale))
        return fail(DSPARK_ERR_INVALID_ARG, "scale must be finite");
    if (!stride_ok(q_ts) || !stride_ok(q_hs) || q_ts % 8 != 0 || q_hs % 8 != 0)
        return fail(DSPARK_ERR_ALIGNMENT, "strides of q must be multiples of 8 elements");
    if (rows > 0 && requests > 0 && (!q || !query_start))
        return fail(DSPARK_ERR_INVALID_ARG, "null q or query_start");
    if (!aligned(q, 16) || !aligned(query_start, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "q must be 16-byte, query_start, scales and error_flags 4-byte aligned");
    p = AttnParams{};
    p.q = static_cast<const uint16_t *>(q);
    p.q_ts = q_ts;
    p.q_hs = q_hs;
    p.num_rows = rows;
    p.cache = static_cast<const unsigned char *>(cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.query_start = query_start;
    p.context_lens = lens;
    p.error_flags = error_flags;
    p.num_blocks = num_blocks;
    p.num_heads = heads;
    p.num_kv_heads = nkv;
    p.group = heads / nkv;
    p.block_size = block_size;
    p.block_magic = block_size > 1 ? UINT64_MAX / (uint64_t)block_size + 1 : 0;
    p.num_requests = requests;
    p.scale = scale;
    const uint64_t hold = test_hold_ns();
    p.test_hold = hold != 0;
    p.wait_ns = hold ? hold : kWaitNs;
    return DSPARK_OK;
}

}  // namespace

extern "C" {

int dspark_rope_table(void *out, int64_t first_position, int64_t num_positions, int rotary_dim, const double *freqs,
                      double amplitude, int out_fp32, cudaStream_t stream)
{
    if (rotary_dim < 2 || rotary_dim > kMaxRotary || rotary_dim % 2 != 0)
        return fail(DSPARK_ERR_UNSUPPORTED_ROTARY_DIM, "rotary_dim %d must be even and in [2, %d]", rotary_dim, kMaxRotary);
    const int64_t most = (int64_t)1 << 31;
    if (first_position < 0 || num_positions < 0 || first_position > most || num_positions > most - first_position)
        return fail(DSPARK_ERR_INVALID_ARG, "positions [%lld, +%lld) not in [0, 2^31)", (long long)first_position,
                    (long long)num_positions);
    if (!std::isfinite((float)amplitude))
        return fail(DSPARK_ERR_INVALID_ARG, "amplitude must be finite in fp32");
    if (!freqs)
        return fail(DSPARK_ERR_INVALID_ARG, "null freqs");
    RopeTableParams p;
    for (int i = 0; i < rotary_dim / 2; i++) {
        if (!std::isfinite(freqs[i]))
            return fail(DSPARK_ERR_INVALID_ARG, "freqs[%d] is not finite", i);
        p.turns[i] = fraction_of_a_turn(freqs[i]);
    }
    if (num_positions == 0)
        return ok();
    if (!out)
        return fail(DSPARK_ERR_INVALID_ARG, "null out");
    if (!aligned(out, 16))
        return fail(DSPARK_ERR_ALIGNMENT, "out must be 16-byte aligned");
    p.out = out;
    p.first = first_position;
    p.count = num_positions;
    p.rotary_dim = rotary_dim;
    p.amplitude = (float)amplitude;
    return launched(launch_rope_table(p, out_fp32 != 0, stream), "rope table");
}

int dspark_rope_kv_insert(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                          int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                          int64_t v_head_stride, void *q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                          void *k_out, int64_t ko_token_stride, int64_t ko_head_stride, const void *cos_sin,
                          int cos_sin_fp32, int64_t max_pos, const int64_t *positions, int64_t num_tokens,
                          int num_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int inverse,
                          const int64_t *slot_mapping, void *kv_cache, int64_t num_blocks, int block_size,
                          int kv_dtype, const float *k_scale, const float *v_scale, unsigned int *error_flags,
                          cudaStream_t stream)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(DSPARK_ERR_INVALID_ARG, "head_dim %d not in {64, 128, 256}", head_dim);
    if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 != 0)
        return fail(DSPARK_ERR_UNSUPPORTED_ROTARY_DIM, "rotary_dim %d must be even and in [2, %d]", rotary_dim, head_dim);
    if (num_heads < 1 || num_kv_heads < 1 || num_heads > (1 << 20) || num_kv_heads > 65535)
        return fail(DSPARK_ERR_INVALID_ARG, "num_heads=%d num_kv_heads=%d out of range", num_heads, num_kv_heads);
    if (num_tokens < 0 || num_tokens > (int64_t)1 << 40)
        return fail(DSPARK_ERR_INVALID_ARG, "num_tokens %lld out of range", (long long)num_tokens);
    if (max_pos < 1)
        return fail(DSPARK_ERR_INVALID_ARG, "max_pos %lld must be >= 1", (long long)max_pos);
    if ((slot_mapping != nullptr) != (kv_cache != nullptr))
        return fail(DSPARK_ERR_INVALID_ARG, "slot_mapping and kv_cache go together (both or neither)");
    const bool insert = slot_mapping != nullptr;
    if (insert) {
        const int st = check_cache(kv_cache, num_blocks, num_kv_heads, block_size, head_dim, kv_dtype);
        if (st != DSPARK_OK)
            return st;
        if (!aligned(slot_mapping, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
            return fail(DSPARK_ERR_ALIGNMENT, "slot_mapping must be 8-byte and scales 4-byte aligned");
    }
    const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride,
                               v_head_stride, qo_token_stride, qo_head_stride, ko_token_stride, ko_head_stride};
    for (int64_t s : strides)
        if (!stride_ok(s))
            return fail(DSPARK_ERR_INVALID_ARG, "stride %lld out of range", (long long)s);
    if (num_tokens == 0)
        return ok();
    if (!q || !k || !q_out || !k_out || !cos_sin || !positions || (insert && !v))
        return fail(DSPARK_ERR_INVALID_ARG, "null q, k, v, q_out, k_out, cos_sin or positions");
    if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(q_out, 2) || !aligned(k_out, 2) ||
        !aligned(cos_sin, 16) || !aligned(positions, 8) || !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "bf16 rows must be 2-byte, cos_sin 16-byte, positions 8-byte aligned");
    RopeInsertParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.q_ts = q_token_stride, p.q_hs = q_head_stride;
    p.k_ts = k_token_stride, p.k_hs = k_head_stride;
    p.v_ts = v_token_stride, p.v_hs = v_head_stride;
    p.qo_ts = qo_token_stride, p.qo_hs = qo_head_stride;
    p.ko_ts = ko_token_stride, p.ko_hs = ko_head_stride;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.cache = static_cast<unsigned char *>(kv_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.error_flags = error_flags;
    p.num_tokens = num_tokens;
    p.max_pos = max_pos;
    p.capacity = insert ? num_blocks * (int64_t)block_size : 0;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary_dim = rotary_dim;
    p.block_size = insert ? block_size : 1;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    p.table_fp32 = cos_sin_fp32 != 0;
    p.fp8 = insert && kv_dtype == DSPARK_KV_FP8_E4M3;
    // 16-byte words: aligned rows of all five tensors, and a lane's 8 dims
    // that rotate together
    p.vec = rotary_dim % (p.interleaved ? 8 : 16) == 0 && aligned(q, 16) && aligned(k, 16) && aligned(q_out, 16) &&
            aligned(k_out, 16) && (!insert || aligned(v, 16));
    for (int i = 0; i < 10; i++)
        if (strides[i] % 8 != 0 && (insert || (i != 4 && i != 5)))
            p.vec = false;
    return launched(launch_rope_insert(p, head_dim, stream), "rope insert");
}

int64_t dspark_tree_attention_workspace(int64_t num_rows, int num_heads, int num_kv_heads, int head_dim,
                                        int num_requests, int kv_dtype)
{
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        !attention_sizes_ok(num_rows, num_heads, num_kv_heads, num_requests) ||
        (kv_dtype != DSPARK_KV_BF16 && kv_dtype != DSPARK_KV_FP8_E4M3)) {
        fail(DSPARK_ERR_INVALID_ARG, "tree attention workspace: invalid sizes");
        return -1;
    }
    if (num_rows == 0 || num_requests == 0)
        return 0;
    cudaError_t e = cudaSuccess;
    const int64_t n = tree_attention_workspace(num_rows, num_heads, num_kv_heads, head_dim, num_requests,
                                               kv_dtype == DSPARK_KV_FP8_E4M3, e);
    if (e != cudaSuccess) {
        launched(e, "tree attention workspace");
        return -1;
    }
    return n;
}

int dspark_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_rows,
                          int num_heads, int num_kv_heads, int head_dim, const void *kv_cache, int64_t num_blocks,
                          int block_size, int kv_dtype, const float *k_scale, const float *v_scale,
                          const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                          const int32_t *query_start, const int32_t *context_lens, int num_requests, int mask_kind,
                          const uint64_t *tree_mask, int mask_words, float scale, void *out, float *lse,
                          void *workspace, int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream)
{
    AttnParams p;
    const int st = check_attention(p, q, q_token_stride, q_head_stride, num_rows, num_heads, num_kv_heads, head_dim,
                                   kv_cache, num_blocks, block_size, kv_dtype, k_scale, v_scale, block_table,
                                   table_stride, table_blocks, query_start, context_lens, num_requests, scale,
                                   error_flags);
    if (st != DSPARK_OK)
        return st;
    if (mask_kind != DSPARK_MASK_DENSE && mask_kind != DSPARK_MASK_CAUSAL && mask_kind != DSPARK_MASK_TREE)
        return fail(DSPARK_ERR_INVALID_ARG, "mask kind %d unknown", mask_kind);
    if (mask_kind == DSPARK_MASK_TREE && (mask_words < 1 || mask_words > (1 << 16)))
        return fail(DSPARK_ERR_INVALID_ARG, "mask_words %d not in [1, 65536]", mask_words);
    if (num_rows == 0 || num_requests == 0)
        return ok();
    if (!out || !lse || (mask_kind == DSPARK_MASK_TREE && !tree_mask))
        return fail(DSPARK_ERR_INVALID_ARG, "null out, lse or tree_mask");
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(tree_mask, 8) || !aligned(workspace, 16))
        return fail(DSPARK_ERR_ALIGNMENT, "out and workspace must be 16-byte, tree_mask 8-byte, lse 4-byte aligned");
    const bool fp8 = kv_dtype == DSPARK_KV_FP8_E4M3;
    cudaError_t e = cudaSuccess;
    const int64_t need = tree_attention_workspace(num_rows, num_heads, num_kv_heads, head_dim, num_requests, fp8, e);
    if (e != cudaSuccess)
        return launched(e, "tree attention");
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(DSPARK_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                    (long long)need);
    p.mask_kind = mask_kind;
    p.tree_mask = tree_mask;
    p.mask_words = mask_words;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.parts = static_cast<float *>(workspace);
    return launched(launch_tree_attention(p, head_dim, fp8, stream), "tree attention");
}

int dspark_attention_weight_accumulate(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t num_rows,
                                       int num_heads, int num_kv_heads, int head_dim, const void *kv_cache,
                                       int64_t num_blocks, int block_size, int kv_dtype, const float *k_scale,
                                       const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                                       const int32_t *query_start, const int32_t *context_lens, int num_requests,
                                       const float *lse, float scale, float decay, float *weights,
                                       int64_t weight_stride, unsigned int *error_flags, cudaStream_t stream)
{
    AttnParams p;
    const int st = check_attention(p, q, q_token_stride, q_head_stride, num_rows, num_heads, num_kv_heads, head_dim,
                                   kv_cache, num_blocks, block_size, kv_dtype, k_scale, nullptr, block_table,
                                   table_stride, table_blocks, query_start, context_lens, num_requests, scale,
                                   error_flags);
    if (st != DSPARK_OK)
        return st;
    if (!std::isfinite(decay))
        return fail(DSPARK_ERR_INVALID_ARG, "decay must be finite");
    if (weight_stride < 0 || weight_stride > INT32_MAX)
        return fail(DSPARK_ERR_INVALID_ARG, "weight_stride %lld out of range", (long long)weight_stride);
    if (num_requests == 0 || weight_stride == 0)
        return ok();
    if (!weights || !query_start || (num_rows > 0 && !lse))
        return fail(DSPARK_ERR_INVALID_ARG, "null weights, query_start or lse");
    if (!aligned(weights, 4) || !aligned(lse, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "weights and lse must be 4-byte aligned");
    p.lse = const_cast<float *>(lse);
    p.weights = weights;
    p.weight_stride = weight_stride;
    p.decay = decay;
    return launched(launch_attention_weight(p, head_dim, kv_dtype == DSPARK_KV_FP8_E4M3, stream), "attention weight");
}

int64_t dspark_kv_evict_workspace(int num_requests, int num_kv_heads, int64_t stride, int64_t budget)
{
    if (!evict_sizes_ok(num_requests, num_kv_heads, stride) || budget < 1) {
        fail(DSPARK_ERR_INVALID_ARG, "evict workspace: invalid sizes");
        return -1;
    }
    // per pair the number of moves, the list of places given up and the list
    // of tokens that move
    const int64_t len = std::max<int64_t>(0, std::min(budget, stride - budget));
    return (int64_t)num_requests * num_kv_heads * (1 + 2 * len) * 4;
}

int dspark_kv_evict(void *kv_cache, int64_t num_blocks, int num_kv_heads, int block_size, int head_dim, int kv_dtype,
                    const int32_t *block_table, int64_t table_stride, int64_t table_blocks,
                    const int32_t *context_lens, int num_requests, const float *weights, const int32_t *positions,
                    float *weights_out, int32_t *positions_out, int64_t stride, const int32_t *seq_lens,
                    int64_t budget, int64_t sinks, int64_t recent, int32_t *new_lens, void *workspace,
                    int64_t workspace_bytes, unsigned int *error_flags, cudaStream_t stream)
{
    int st = check_cache(kv_cache, num_blocks, num_kv_heads, block_size, head_dim, kv_dtype);
    if (st != DSPARK_OK)
        return st;
    if ((st = check_table(block_table, table_stride, table_blocks, num_requests, context_lens)) != DSPARK_OK)
        return st;
    if (stride < 0 || stride > (int64_t)INT32_MAX - 1024)
        return fail(DSPARK_ERR_INVALID_ARG, "stride %lld out of range", (long long)stride);
    if (budget < 1 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return fail(DSPARK_ERR_INVALID_ARG, "budget %lld, sinks %lld, recent %lld: 1 <= sinks + recent <= budget wanted",
                    (long long)budget, (long long)sinks, (long long)recent);
    if (!evict_sizes_ok(num_requests, num_kv_heads, stride))
        return fail(DSPARK_ERR_INVALID_ARG, "%d requests of %d heads: too many", num_requests, num_kv_heads);
    if (num_requests == 0)
        return ok();
    if (!new_lens || !seq_lens || (stride > 0 && (!weights || !positions || !weights_out || !positions_out)))
        return fail(DSPARK_ERR_INVALID_ARG, "null weights, positions, seq_lens or an output");
    if (!aligned(weights, 4) || !aligned(positions, 4) || !aligned(weights_out, 4) || !aligned(positions_out, 4) ||
        !aligned(new_lens, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 16) || !aligned(error_flags, 4))
        return fail(DSPARK_ERR_ALIGNMENT, "workspace must be 16-byte, the other buffers 4-byte aligned");
    if (overlap_partly(new_lens, context_lens, num_requests) || overlap_partly(new_lens, seq_lens, num_requests))
        return fail(DSPARK_ERR_INVALID_ARG, "new_lens overlaps context_lens or seq_lens without being one of them");
    // weights that change while they are ranked would give lists longer than the workspace's
    const int64_t entries = (int64_t)num_requests * num_kv_heads * stride;
    if (overlap_partly(weights_out, weights, entries) || overlap_partly(positions_out, positions, entries))
        return fail(DSPARK_ERR_INVALID_ARG, "weights_out or positions_out overlaps its input without being it");
    if (entries > 0 && (weights_out == (const void *)positions || overlap_partly(weights_out, positions, entries) ||
                        positions_out == (const void *)weights || overlap_partly(positions_out, weights, entries) ||
                        weights_out == (void *)positions_out || overlap_partly(weights_out, positions_out, entries)))
        return fail(DSPARK_ERR_INVALID_ARG, "weights and positions overlap");
    const int64_t need = dspark_kv_evict_workspace(num_requests, num_kv_heads, stride, budget);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(DSPARK_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                    (long long)need);
    EvictParams p{};
    p.cache = static_cast<unsigned char *>(kv_cache);
    p.table = block_table;
    p.table_stride = table_stride;
    p.table_blocks = usable_blocks(table_blocks, block_size);
    p.context_lens = context_lens;
    p.seq_lens = seq_lens;
    p.weights = weights;
    p.positions = positions;
    p.weights_out = weights_out;
    p.positions_out = positions_out;
    p.new_lens = new_lens;
    p.counts = static_cast<int32_t *>(workspace);
    p.lists = p.counts + (int64_t)num_requests * num_kv_heads;
    p.error_flags = error_flags;
    p.num_blocks = num_blocks;
    p.stride = stride;
    p.list_len = std::max<int64_t>(0, std::min(budget, stride - budget));
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    p.num_requests = num_requests;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.row_bytes = 2 * head_dim * (kv_dtype == DSPARK_KV_FP8_E4M3 ? 1 : 2);
    return launched(launch_kv_evict(p, stream), "evict");
}

}  // extern "C"
