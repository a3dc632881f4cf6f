// Pages of the cache: the accepted path's K|V moved together, and pages of the
// pool shared, copied, reserved and freed (sm_103a).
//
// None of it computes: what bounds it is the chain of dependent loads (length,
// path, block table, rows) and a launch, then the rows' bytes.
#include <cooperative_groups.h>

#include "ctx_kv_internal.h"
#include "draft_step_internal.h"
#include "page_scale.cuh"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ the accepted path

constexpr int kMoves = 256;  // moves whose rows are looked up at once
constexpr int kDeep = 8;     // loads in flight per thread

// One (request, layer) per CTA.  A thread has one 16-byte column of a head's rows
// (several, where a token has more of them than the CTA threads) and moves it
// through the path in order.  Paths ascend and never move a row back, so no
// row is written before it has been read: a row is written at or before the place
// it comes from, and later moves read from behind that.  Batches of kDeep loads
// keep that order.
//
// Page-scaled: page by page that rows move into.  Scales are read as they were:
// rows come from the page itself or later ones, whose scales change later; a
// page's own is written when all its rows are done.
template <bool SCALED>
__global__ void __launch_bounds__(256) compact_kernel(const __grid_constant__ CompactParams p)
{
    __shared__ int64_t src_row[kMoves], dst_row[kMoves];  // (page * heads * block_size + offset), < 0: does not move
    __shared__ int64_t src_page[kMoves];
    pdl_enter();
    const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, H = p.num_kv_heads, bs = p.block_size;
    unsigned flags = 0;
    const int ctx = __ldg(p.context_lens + b), count = __ldg(p.counts + b);
    const int32_t *path = p.rows + b * p.rows_stride, *table = p.table + b * p.table_stride;
    const int64_t room = p.table_blocks * bs;
    // the path: ascending, at or behind where it moves to, inside the table
    bool bad = ctx < 0 || count < 0 || count > p.width || (int64_t)ctx + p.first + count > room;
    if (!bad)
        for (int j = tid; j < count; j += blockDim.x) {
            const int r = __ldg(path + j);
            bad |= r < p.first + j || (j && __ldg(path + j - 1) >= r) || (int64_t)ctx + r >= room;
        }
    bad = __syncthreads_or(bad);
    if (layer == 0 && tid == 0 && p.new_lens)
        p.new_lens[b] = bad ? ctx : ctx + p.first + count;
    if (bad) {
        if (tid == 0 && p.error_flags)
            atomicOr(p.error_flags, kFlagLength);
        return;
    }
    unsigned char *cache = p.layers.cache[layer];
    int8_t *scales = SCALED ? p.layers.scales[layer] : nullptr;
    const int words = p.row_bytes / 16, columns = H * words;
    const int64_t head_bytes = (int64_t)bs * p.row_bytes;

    auto look_up = [&](int j0, int n) {  // moves j0 .. j0 + n
        for (int j = tid; j < n; j += blockDim.x) {
            const int s = ctx + __ldg(path + j0 + j), d = ctx + p.first + j0 + j;
            int64_t sr = -1, dr = -1, sp = -1;
            if (s != d) {
                sp = __ldg(table + s / bs);
                const int64_t dp = __ldg(table + d / bs);
                if (sp < 0 || sp >= p.num_blocks || dp < 0 || dp >= p.num_blocks)
                    flags |= kFlagBlockRange, sp = -1;
                else
                    sr = sp * H * bs + s % bs, dr = dp * H * bs + d % bs;
            }
            src_row[j] = sr, dst_row[j] = dr;
            src_page[j] = sp;
        }
        __syncthreads();
    };

    if constexpr (!SCALED) {
        for (int j0 = 0; j0 < count; j0 += kMoves) {
            const int n = min(kMoves, count - j0);
            look_up(j0, n);
            for (int x = tid; x < columns; x += blockDim.x) {
                const int h = x / words;
                unsigned char *column = cache + h * head_bytes + (x - h * words) * 16;
                for (int j = 0; j < n; j += kDeep) {
                    uint4 v[kDeep];
#pragma unroll
                    for (int k = 0; k < kDeep; k++)
                        if (j + k < n && src_row[j + k] >= 0)
                            v[k] = *reinterpret_cast<const uint4 *>(column + src_row[j + k] * p.row_bytes);
#pragma unroll
                    for (int k = 0; k < kDeep; k++)
                        if (j + k < n && src_row[j + k] >= 0)
                            *reinterpret_cast<uint4 *>(column + dst_row[j + k] * p.row_bytes) = v[k];
                }
            }
            __syncthreads();
        }
    } else {
        const int d0 = ctx + p.first;  // places [d0, d0 + count) are written
        for (int j0 = 0; j0 < count;) {
            const int blk = (d0 + j0) / bs;
            const int n = (int)min((int64_t)count - j0, (int64_t)(blk + 1) * bs - (d0 + j0));  // moves into this page
            const int64_t page = __ldg(table + blk);
            // the scale that the page needs, over all moves into it: a thread per (head, part)
            const bool fits = n <= kMoves;
            if (fits)
                look_up(j0, n);
            for (int m0 = 0; m0 < n; m0 += kMoves) {
                const int m = min(kMoves, n - m0);
                if (!fits)
                    look_up(j0 + m0, m);
                for (int x = tid; x < columns; x += blockDim.x) {
                    const int h = x / words, w = x - h * words, part = w >= words / 2;
                    unsigned char *column = cache + h * head_bytes + w * 16;
                    if (page < 0 || page >= p.num_blocks)
                        continue;  // its moves are marked
                    const int own = page_exponent(scales, page, H, h, part);
                    int top = own;
                    if (fits) {
                        for (int k = 0; k < m; k++)
                            if (src_page[k] >= 0)
                                top = max(top, page_exponent(scales, src_page[k], H, h, part));
                    } else {
                        for (int k = 0; k < n; k++) {
                            const int s = ctx + __ldg(path + j0 + k);
                            const int64_t sp = __ldg(table + s / bs);
                            if (s != d0 + j0 + k && sp >= 0 && sp < p.num_blocks)
                                top = max(top, page_exponent(scales, sp, H, h, part));
                        }
                    }
                    if (m0 == 0 && top > own) {
                        // all that the page holds, at its new scale
                        const uint32_t f = half2_power(top - own);
                        unsigned char *at = column + page * H * head_bytes;
                        for (int o = 0; o < bs; o += kDeep) {
                            uint4 v[kDeep];
#pragma unroll
                            for (int k = 0; k < kDeep; k++)
                                if (o + k < bs)
                                    v[k] = *reinterpret_cast<const uint4 *>(at + (int64_t)(o + k) * p.row_bytes);
#pragma unroll
                            for (int k = 0; k < kDeep; k++)
                                if (o + k < bs)
                                    *reinterpret_cast<uint4 *>(at + (int64_t)(o + k) * p.row_bytes) = scale_codes(v[k], f);
                        }
                    }
                    for (int j = 0; j < m; j += kDeep) {
                        uint4 v[kDeep];
                        uint32_t f[kDeep];
#pragma unroll
                        for (int k = 0; k < kDeep; k++)
                            if (j + k < m && src_row[j + k] >= 0) {
                                v[k] = *reinterpret_cast<const uint4 *>(column + src_row[j + k] * p.row_bytes);
                                // rows of this page have its new scale already
                                f[k] = half2_power(src_page[j + k] == page ? 0 : top - page_exponent(scales, src_page[j + k], H, h, part));
                            }
#pragma unroll
                        for (int k = 0; k < kDeep; k++)
                            if (j + k < m && src_row[j + k] >= 0)
                                *reinterpret_cast<uint4 *>(column + dst_row[j + k] * p.row_bytes) = f[k] == 0x3c003c00u ? v[k] : scale_codes(v[k], f[k]);
                    }
                }
                __syncthreads();  // the lists are free, and everyone has read the scales
            }
            if (page >= 0 && page < p.num_blocks)
                for (int x = tid; x < 2 * H; x += blockDim.x) {
                    int top = page_exponent(scales, page, H, x >> 1, x & 1);
                    const int own = top;
                    for (int k = 0; k < n; k++) {
                        const int s = ctx + __ldg(path + j0 + k);
                        const int64_t sp = __ldg(table + s / bs);
                        if (s != d0 + j0 + k && sp >= 0 && sp < p.num_blocks && sp != page)
                            top = max(top, page_exponent(scales, sp, H, x >> 1, x & 1));
                    }
                    if (top != own)
                        scales[(page * H + (x >> 1)) * 2 + (x & 1)] = (int8_t)top;
                }
            j0 += n;
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && (tid & 31) == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

// ------------------------------------------------------------------ the pool

constexpr int kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32, kPoolCtas = 8;

struct PoolShared {
    int sums[kPoolCtas], warps[kPoolWarps];
    int64_t wide[kPoolWarps];
};

// This thread's exclusive prefix of x over the CTA, and the CTA's sum.
template <typename T>
__device__ __forceinline__ T cta_prefix(T x, T &sum, T *warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T up = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d)
            up += y;
    }
    __syncthreads();  // warps[] is free
    if (lane == 31)
        warps[warp] = up;
    __syncthreads();
    T t = warps[lane], all = t;
    t = lane < warp ? t : 0;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        t += __shfl_xor_sync(0xffffffffu, t, d);
        all += __shfl_xor_sync(0xffffffffu, all, d);
    }
    sum = all;
    return t + up - x;
}

// Counts the free pages of this CTA's share [lo, hi) of the pool; returns how many
// the CTAs before it have, `free` all of the cluster's.
__device__ __forceinline__ int count_free(cg::cluster_group &cluster, const int32_t *refs, int64_t lo, int64_t hi, int &free, PoolShared &s)
{
    int mine = 0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kPoolThreads)
        mine += __ldcg(refs + i) == 0;
    int sum;
    cta_prefix(mine, sum, s.warps);
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    if ((int)threadIdx.x < nc)
        cluster.map_shared_rank(&s.sums[0], threadIdx.x)[rank] = sum;
    cluster.sync();
    int before = 0;
    free = 0;
    for (int r = 0; r < nc; r++) {
        before += r < rank ? s.sums[r] : 0;
        free += s.sums[r];
    }
    return before;
}

// give(k, page) for the free pages of [lo, hi) in rising order, k from `before` on, below `most`
template <typename F>
__device__ __forceinline__ void each_free(const int32_t *refs, int64_t lo, int64_t hi, int before, int most, PoolShared &s, F give)
{
    for (int64_t i0 = lo; i0 < hi && before < most; i0 += kPoolThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool is = i < hi && __ldcg(refs + i) == 0;
        int sum;
        const int k = before + cta_prefix((int)is, sum, s.warps);
        if (is && k < most)
            give(k, (int)i);
        before += sum;
    }
}

// Pairs, free pages and everything but the pages' contents, by one cluster (the
// free pages' ranks need all of the pool; 65,536 pages are 32 KB per CTA).
__global__ void __launch_bounds__(kPoolThreads, 1) fork_kernel(const __grid_constant__ ForkParams p)
{
    __shared__ PoolShared sh;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nc = (int)cluster.num_blocks(), tid = threadIdx.x, bs = p.block_size;
    unsigned flags = 0;
    const int64_t share = (p.num_blocks + nc - 1) / nc, lo = min(p.num_blocks, share * rank), hi = min(p.num_blocks, lo + share);

    // ---- the pairs: which are sound, what they copy (each CTA a part; z: the pair's state)
    for (int i = rank * kPoolThreads + tid; i < p.num_pairs; i += nc * kPoolThreads) {
        const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
        bool ok = s >= 0 && s < p.num_rows && d >= 0 && d < p.num_rows;
        int old = -1, tail = 0;
        if (ok) {
            const int64_t len = p.lens[s], held = p.pages[s];
            ok = p.pages[d] == 0 && len >= 0 && held >= 0 && held <= p.table_blocks && len <= held * bs;
            if (ok) {
                for (int k = 0; k < p.num_pairs; k++)
                    ok &= __ldg(p.src + k) != d && (k >= i || __ldg(p.dst + k) != d);
                tail = (int)(len % bs);
                if (tail) {
                    old = p.table[s * p.table_stride + len / bs];
                    if (ok && (old < 0 || old >= p.num_blocks)) {
                        flags |= kFlagBlockRange;
                        ok = false;
                        tail = -1;
                    }
                }
            }
        }
        if (!ok && tail >= 0)
            flags |= kFlagLength;
        p.copies[i] = make_int4(old, -1, ok ? tail : 0, ok);
    }
    cluster.sync();  // all of `copies` is there; every CTA of the cluster runs

    // ---- the k-th free page goes to the k-th sound pair that needs one (found by every CTA for itself)
    int free;
    const int before = count_free(cluster, p.refs, lo, hi, free, sh);
    int need = 0;
    for (int i0 = 0; i0 < p.num_pairs; i0 += kPoolThreads) {
        const int i = i0 + tid;
        const bool needs = i < p.num_pairs && __ldcg(&p.copies[i]).z > 0;
        int sum;
        cta_prefix((int)needs, sum, sh.warps);
        need += sum;
    }
    cluster.sync();  // nobody reads `copies` as it was any more
    // ranks of the pairs: as y = -2 - rank, by the first CTA; then the pages' owners look for them
    if (rank == 0) {
        int at = 0;
        for (int i0 = 0; i0 < p.num_pairs; i0 += kPoolThreads) {
            const int i = i0 + tid;
            const bool needs = i < p.num_pairs && __ldcg(&p.copies[i]).z > 0;
            int sum;
            const int k = at + cta_prefix((int)needs, sum, sh.warps);
            if (needs) {
                p.copies[i].y = -1;
                p.copies[p.num_pairs + k].x = i;  // the k-th pair in need
                if (k >= free) {                  // none left for it
                    flags |= kFlagPages;
                    p.copies[i].z = 0;
                    p.copies[i].w = 0;
                }
            }
            at += sum;
        }
    }
    cluster.sync();
    each_free(p.refs, lo, hi, before, min(need, free), sh, [&](int k, int page) {
        const int i = __ldcg(&p.copies[p.num_pairs + k].x);
        p.copies[i].y = page;
    });
    cluster.sync();

    // ---- table rows, references, lengths: the pairs' entries over all threads
    const int threads = nc * kPoolThreads, me = rank * kPoolThreads + tid;
    // as many threads to a pair as there are for each, at least a warp
    int per = 32;
    while (per * 2 * p.num_pairs <= threads)
        per *= 2;
    for (int i = me / per; i < p.num_pairs; i += threads / per) {
        const int4 c = __ldcg(&p.copies[i]);
        if (!c.w)
            continue;
        const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
        const int len = p.lens[s], full = len / bs;
        const int32_t *from = p.table + s * p.table_stride;
        int32_t *to = p.table + d * p.table_stride;
        for (int k = me % per; k < full; k += per) {
            const int page = from[k];
            to[k] = page;
            if (page >= 0 && page < p.num_blocks)
                atomicAdd(p.refs + page, 1);
            else
                flags |= kFlagBlockRange;
        }
        if (me % per == 0) {
            if (c.z > 0) {
                to[full] = c.y;
                p.refs[c.y] = 1;
            }
            p.pages[d] = full + (c.z > 0);
            p.lens[d] = len;
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && (tid & 31) == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

// One (pair, layer, head) per CTA: the tokens of a page of that head are one run of bytes.
__global__ void __launch_bounds__(128) page_copy_kernel(const __grid_constant__ PageCopyParams p)
{
    pdl_enter();
    const int4 c = p.copies[blockIdx.x];
    if (c.z <= 0)
        return;
    const int layer = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
    const int64_t page_bytes = (int64_t)p.block_size * p.row_bytes;
    const unsigned char *from = p.layers.cache[layer] + ((int64_t)c.x * p.num_kv_heads + h) * page_bytes;
    unsigned char *to = p.layers.cache[layer] + ((int64_t)c.y * p.num_kv_heads + h) * page_bytes;
    const int64_t words = (int64_t)c.z * (p.row_bytes / 16);
    for (int64_t i0 = tid; i0 < words; i0 += 128 * kDeep) {
        uint4 v[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; k++)
            if (i0 + 128 * k < words)
                v[k] = *reinterpret_cast<const uint4 *>(from + (i0 + 128 * k) * 16);
#pragma unroll
        for (int k = 0; k < kDeep; k++)
            if (i0 + 128 * k < words)
                *reinterpret_cast<uint4 *>(to + (i0 + 128 * k) * 16) = v[k];
    }
    if (p.scaled && tid < 2)
        p.layers.scales[layer][((int64_t)c.y * p.num_kv_heads + h) * 2 + tid] =
            p.layers.scales[layer][((int64_t)c.x * p.num_kv_heads + h) * 2 + tid];
}

// Entries given back, then pages taken, by one cluster.
__global__ void __launch_bounds__(kPoolThreads, 1) resize_kernel(const __grid_constant__ ResizeParams p)
{
    __shared__ PoolShared sh;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nc = (int)cluster.num_blocks(), tid = threadIdx.x, bs = p.block_size;
    unsigned flags = 0;
    const int64_t share = (p.num_blocks + nc - 1) / nc, lo = min(p.num_blocks, share * rank), hi = min(p.num_blocks, lo + share);
    // pages that row r holds and wants, whether both fit the table
    auto row = [&](int r, int &have, int &want) {
        have = __ldcg(p.pages + r);
        const int tokens = __ldg(p.tokens + r);
        want = tokens / bs + (tokens % bs > 0);
        return have >= 0 && have <= p.table_blocks && tokens >= 0 && want <= p.table_blocks;
    };

    // ---- back to the pool; p.before holds the rows' needs for now
    const int threads = nc * kPoolThreads, me = rank * kPoolThreads + tid;
    int per = 32;
    while (per * 2 * (int64_t)p.num_rows <= threads)
        per *= 2;
    for (int r = me / per; r < p.num_rows; r += threads / per) {
        int have, want;
        const bool ok = row(r, have, want);
        if (!ok)
            flags |= kFlagLength;
        int32_t *entries = p.table + r * p.table_stride;
        if (ok)
            for (int k = want + me % per; k < have; k += per) {
                const int page = entries[k];
                entries[k] = -1;
                if (page < 0 || page >= p.num_blocks) {
                    flags |= kFlagBlockRange;
                } else if (atomicSub(p.refs + page, 1) <= 0) {
                    atomicAdd(p.refs + page, 1);  // nobody held it
                    flags |= kFlagRefs;
                }
            }
        __syncwarp();  // (per >= 32: a row's threads are whole warps)
        if (me % per == 0)
            p.before[r] = ok && want > have ? want - have : 0;
    }
    __threadfence();
    cluster.sync();

    int free;
    const int before = count_free(cluster, p.refs, lo, hi, free, sh);
    // ---- the needs of the rows before each, by the first CTA
    if (rank == 0) {
        int64_t at = 0;
        for (int r0 = 0; r0 < p.num_rows; r0 += kPoolThreads) {
            const int r = r0 + tid;
            const int64_t need = r < p.num_rows ? __ldcg(p.before + r) : 0;
            int64_t sum;
            const int64_t k = cta_prefix(need, sum, sh.wide);
            if (r < p.num_rows)
                p.before[r] = (int32_t)min(at + k, (int64_t)INT32_MAX);  // more than any pool has
            at += sum;
        }
        if (tid == 0)
            p.before[p.num_rows] = (int32_t)min(at, (int64_t)INT32_MAX);
    }
    cluster.sync();
    const int need = __ldcg(p.before + p.num_rows);
    each_free(p.refs, lo, hi, before, min(need, free), sh, [&](int k, int page) {
        // the last row with before <= k: rows that need none share their `before` with the next
        int a = 0, z = p.num_rows;
        while (z - a > 1) {
            const int m = (a + z) >> 1;
            if (__ldcg(p.before + m) <= k)
                a = m;
            else
                z = m;
        }
        const int first = __ldcg(p.before + a);
        if (__ldcg(p.before + a + 1) > free)
            return;  // not all of what the row asks for is there
        int have, want;
        row(a, have, want);
        p.table[a * p.table_stride + have + (k - first)] = page;
        p.refs[page] = 1;
    });
    cluster.sync();  // everyone has read `pages`
    for (int r = me; r < p.num_rows; r += threads) {
        int have, want;
        if (!row(r, have, want) || have == want)
            continue;
        if (want > have && __ldcg(p.before + r + 1) > free) {
            flags |= kFlagPages;
            continue;
        }
        p.pages[r] = want;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && (tid & 31) == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

}  // namespace

cudaError_t launch_compact(const CompactParams &p, bool scaled, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.num_requests, (unsigned)p.num_layers);
    return scaled ? launch_pdl_grid(compact_kernel<true>, grid, 256, 0, 0, stream, p)
                  : launch_pdl_grid(compact_kernel<false>, grid, 256, 0, 0, stream, p);
}

cudaError_t launch_fork(const ForkParams &p, cudaStream_t stream)
{
    return launch_pdl_grid(fork_kernel, dim3(kPoolCtas), kPoolThreads, 0, kPoolCtas, stream, p);
}

cudaError_t launch_page_copies(const PageCopyParams &p, cudaStream_t stream)
{
    return launch_pdl_grid(page_copy_kernel, dim3((unsigned)p.num_pairs, (unsigned)p.num_layers, (unsigned)p.num_kv_heads), 128, 0, 0,
                           stream, p);
}

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t stream)
{
    return launch_pdl_grid(resize_kernel, dim3(kPoolCtas), kPoolThreads, 0, kPoolCtas, stream, p);
}

}  // namespace dspark
