// Pages of the cache: the accepted path's K|V moved together, and pages of the
// pool shared, copied, reserved and freed (sm_103a).
//
// None of it computes: what bounds it is the chain of dependent loads (length,
// path, block table, rows) and a launch, then the rows' bytes.  Measured: the
// accepted path of one request in five layers 2.4 us, of 64 in page-scaled caches
// 7.4 us; three forks of one request (the last page copied in five layers) 9.9 us, 64
// forks from a pool of 65,536 pages 13 us, pages given back and taken for 160 rows
// there 19 us, of which four or five cluster barriers are half.
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

// One cluster does a call's bookkeeping: the k-th free page is known only with all
// pages before it counted.  A thread has a run of the pool to itself (4 to 16 pages
// up to 131,072), loads it once, as 16-byte words, and keeps which are free; a
// prefix over the CTA and one exchange over the cluster number them.  Small pools take
// fewer CTAs, whose barriers cost less.
constexpr int kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32, kPoolCtas = 8;
constexpr int kRun = 16;  // pages that a thread keeps in registers at once

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

// This thread's run of the pool, and its free pages in it.
struct Run {
    int64_t lo, hi;
    bool wide;  // 16-byte loads

    __device__ __forceinline__ Run(cg::cluster_group &cluster, const int32_t *refs, int64_t pages)
    {
        const int64_t threads = (int64_t)cluster.num_blocks() * kPoolThreads, me = (int64_t)cluster.block_rank() * kPoolThreads + threadIdx.x;
        const int64_t each = ((pages + threads - 1) / threads + 3) / 4 * 4;
        lo = min(pages, each * me), hi = min(pages, lo + each);
        wide = (reinterpret_cast<uintptr_t>(refs) & 15) == 0;
    }
    // calls f(i, whether pages i .. i + kRun are free, a bit each) for the run; REPAIR: numbers below 0 become 0 (true if there were any)
    template <bool REPAIR, typename F>
    __device__ __forceinline__ bool each(int32_t *refs, F f) const
    {
        bool below = false;
        for (int64_t i = lo; i < hi; i += kRun) {
            int v[kRun];
            if (wide && i + kRun <= hi) {
#pragma unroll
                for (int k = 0; k < kRun; k += 4) {
                    const int4 x = __ldcg(reinterpret_cast<const int4 *>(refs + i + k));
                    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < kRun; k++)
                    v[k] = i + k < hi ? __ldcg(refs + i + k) : 1;
            }
            unsigned bits = 0;
#pragma unroll
            for (int k = 0; k < kRun; k++) {
                bits |= (v[k] == 0 || (REPAIR && v[k] < 0) ? 1u : 0u) << k;
                if (REPAIR && v[k] < 0) {
                    refs[i + k] = 0;
                    below = true;
                }
            }
            f(i, bits);
        }
        return below;
    }
};

// Counts the free pages: this thread's rank of its first, `free` of them all.
// `first` keeps the first kRun pages' bits.  A cluster barrier.
template <bool REPAIR>
__device__ __forceinline__ int rank_free(cg::cluster_group &cluster, const Run &run, int32_t *refs, unsigned &first, int &free, bool &below,
                                         PoolShared &s)
{
    int mine = 0;
    first = 0;
    below = run.each<REPAIR>(refs, [&](int64_t i, unsigned bits) {
        mine += __popc(bits);
        if (i == run.lo)
            first = bits;
    });
    int sum;
    int before = cta_prefix(mine, sum, s.warps);
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    if ((int)threadIdx.x < nc)
        cluster.map_shared_rank(&s.sums[0], threadIdx.x)[rank] = sum;
    cluster.sync();
    free = 0;
    for (int r = 0; r < nc; r++) {
        before += r < rank ? s.sums[r] : 0;
        free += s.sums[r];
    }
    return before;
}

// list[k] = the k-th free page, for k < most
__device__ __forceinline__ void list_free(const Run &run, int32_t *refs, unsigned first, int rank, int most, int32_t *list)
{
    if (run.hi <= run.lo || rank >= most)
        return;
    auto put = [&](int64_t i, unsigned bits) {
        for (; bits && rank < most; bits &= bits - 1)
            list[rank++] = (int32_t)(i + __ffs(bits) - 1);
    };
    if (run.hi - run.lo <= kRun)
        put(run.lo, first);
    else
        run.each<false>(refs, put);
}

// Threads that share a row (or pair) where there are so many: whole warps.
__device__ __forceinline__ int threads_per(int rows, int threads)
{
    int per = 32;
    while (per * 2 * (int64_t)rows <= threads)
        per *= 2;
    return per;
}

// Pairs, free pages and everything but the pages' contents.
__global__ void __launch_bounds__(kPoolThreads, 1) fork_kernel(const __grid_constant__ ForkParams p)
{
    __shared__ PoolShared sh;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nc = (int)cluster.num_blocks(), tid = threadIdx.x, bs = p.block_size;
    const int threads = nc * kPoolThreads, me = rank * kPoolThreads + tid;
    unsigned flags = 0;

    // ---- the pairs: which are sound (w), the page that they copy (x) and its tokens (z)
    for (int i = me; i < p.num_pairs; i += threads) {
        const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
        bool ok = s >= 0 && s < p.num_rows && d >= 0 && d < p.num_rows, bad_page = false;
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
                    bad_page = ok && (old < 0 || old >= p.num_blocks);
                }
            }
        }
        if (!ok || bad_page)
            flags |= bad_page ? kFlagBlockRange : kFlagLength;
        ok = ok && !bad_page;
        p.copies[i] = make_int4(old, -1, ok ? tail : 0, ok);
    }
    cluster.sync();  // all of `copies` is there; every CTA of the cluster runs

    // ---- the k-th free page goes to the k-th sound pair in need
    const Run run(cluster, p.refs, p.num_blocks);
    unsigned first;
    int free;
    bool below;
    const int at = rank_free<false>(cluster, run, p.refs, first, free, below, sh);
    list_free(run, p.refs, first, at, min(free, p.num_pairs), p.free_list);
    cluster.sync();
    if (rank == 0) {
        int before = 0;
        for (int i0 = 0; i0 < p.num_pairs; i0 += kPoolThreads) {
            const int i = i0 + tid;
            const bool needs = i < p.num_pairs && __ldcg(&p.copies[i]).z > 0;
            int sum;
            const int k = before + cta_prefix((int)needs, sum, sh.warps);
            if (needs) {
                if (k < free) {
                    p.copies[i].y = __ldcg(p.free_list + k);
                } else {
                    flags |= kFlagPages;
                    p.copies[i].z = 0;
                    p.copies[i].w = 0;
                }
            }
            before += sum;
        }
    }
    cluster.sync();

    // ---- table rows, references, lengths
    const int per = threads_per(p.num_pairs, threads);
    for (int i = me / per; i < p.num_pairs; i += threads / per) {
        const int4 c = __ldcg(&p.copies[i]);
        if (!c.w)
            continue;
        const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
        const int len = p.lens[s], full = len / bs;
        const int32_t *from = p.table + s * p.table_stride;
        int32_t *to = p.table + d * p.table_stride;
#pragma unroll 4
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

// Entries given back, then pages taken.
__global__ void __launch_bounds__(kPoolThreads, 1) resize_kernel(const __grid_constant__ ResizeParams p)
{
    __shared__ PoolShared sh;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nc = (int)cluster.num_blocks(), tid = threadIdx.x, bs = p.block_size;
    const int threads = nc * kPoolThreads, me = rank * kPoolThreads + tid;
    unsigned flags = 0;
    // pages that row r holds and wants, whether both fit the table
    auto row = [&](int r, int &have, int &want) {
        have = p.pages[r];
        const int tokens = __ldg(p.tokens + r);
        want = tokens / bs + (tokens % bs > 0);
        return have >= 0 && have <= p.table_blocks && tokens >= 0 && want <= p.table_blocks;
    };

    // ---- back to the pool (nothing waits for the counts: one that falls below 0
    // is put right where the pool is read); what each row asks for
    const int per = threads_per(p.num_rows, threads);
    for (int r = me / per; r < p.num_rows; r += threads / per) {
        int have, want;
        const bool ok = row(r, have, want);
        if (!ok)
            flags |= kFlagLength;
        int32_t *entries = p.table + r * p.table_stride;
        if (ok)
#pragma unroll 4
            for (int k = want + me % per; k < have; k += per) {
                const int page = entries[k];
                entries[k] = -1;
                if (page >= 0 && page < p.num_blocks)
                    atomicSub(p.refs + page, 1);
                else
                    flags |= kFlagBlockRange;
            }
        if (me % per == 0)
            p.before[r] = ok && want > have ? want - have : 0;
    }
    cluster.sync();

    // ---- the first CTA sums the rows' needs while all count the pool
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
    const Run run(cluster, p.refs, p.num_blocks);
    unsigned first;
    int free;
    bool below;
    const int at = rank_free<true>(cluster, run, p.refs, first, free, below, sh);
    if (below)
        flags |= kFlagRefs;
    list_free(run, p.refs, first, at, min(free, __ldcg(p.before + p.num_rows)), p.free_list);
    cluster.sync();

    // ---- rows served in their order, as far as the pages go
    for (int r = me / per; r < p.num_rows; r += threads / per) {
        int have, want;
        const bool ok = row(r, have, want);
        const int k0 = __ldcg(p.before + r), k1 = __ldcg(p.before + r + 1);
        const bool served = ok && want > have && k1 <= free;
        if (served) {
            int32_t *entries = p.table + r * p.table_stride;
#pragma unroll 4
            for (int k = me % per; k < want - have; k += per) {
                const int page = __ldcg(p.free_list + k0 + k);
                entries[have + k] = page;
                p.refs[page] = 1;
            }
        }
        if (ok && want > have && !served)
            flags |= kFlagPages;
    }
    cluster.sync();  // every warp has read `pages`
    for (int r = me; r < p.num_rows; r += threads) {
        int have, want;
        if (row(r, have, want) && have != want && (want < have || __ldcg(p.before + r + 1) <= free))
            p.pages[r] = want;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && (tid & 31) == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

// CTAs of the cluster: 8 pages a thread, so that they are loaded at once.
int pool_ctas(int64_t pages)
{
    int nc = 1;
    while (nc < kPoolCtas && pages > (int64_t)nc * kPoolThreads * 8)
        nc *= 2;
    return nc;
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
    const int nc = pool_ctas(p.num_blocks);
    return launch_pdl_grid(fork_kernel, dim3((unsigned)nc), kPoolThreads, 0, nc, stream, p);
}

cudaError_t launch_page_copies(const PageCopyParams &p, cudaStream_t stream)
{
    return launch_pdl_grid(page_copy_kernel, dim3((unsigned)p.num_pairs, (unsigned)p.num_layers, (unsigned)p.num_kv_heads), 128, 0, 0,
                           stream, p);
}

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t stream)
{
    const int nc = pool_ctas(p.num_blocks);
    return launch_pdl_grid(resize_kernel, dim3((unsigned)nc), kPoolThreads, 0, nc, stream, p);
}

}  // namespace dspark
