// Verification of drafted tokens against the target's probabilities (sm_103a).
//
// Mathematics.  Rejections leave R_0 = p, R_{k+1} = max(R_k - Z_k q_k, 0) of the
// target's distribution, Z_k = sum R_k.  q_k is q, or q without the rejected
// children divided by what is left, 1 - Q_k.  Since max(max(a - b, 0) - c, 0) =
// max(a - b - c, 0) for c >= 0, R_k = max(p - S_k q, 0) with one scalar, S_0 = 0,
// S_{k+1} = S_k + Z_k / (1 - Q_k): nothing of a vocabulary's length is stored,
// each round is a pass over one row of p and of q.  (A rejected child x has
// R_k(x) <= u q_k(x) Z_k < q_k(x) Z_k, so it is 0 from then on by itself.)
// The children's p and q are single entries, read all at once beforehand; a chain
// needs no sums before its last row.
//
// Sums are integers in units of 2^-46: entries are rounded to them once (those
// below 2^-23 lose bits), sums are exact and in any order the same.  An entry
// becomes two integers of 23 bits by additions of 2^23 in fp32 (four paired
// operations at the full rate; a conversion to 64 bits runs at a small part of it:
// 44 us against 21 for 64 draws from 131,072 tokens).  The token
// drawn is a whole number that a user compares with one drawn in 64-bit floating
// point: with fp32 terms a rounding of 2^-26 in a heavy entry moves the border of
// every one behind it, which changes one token in some hundreds over a vocabulary
// of 2^17.
//
// Layout.  A cluster of 1 to 16 CTAs per request, each warp with a contiguous
// piece of the vocabulary; all CTAs walk the tree alike (it is the same for
// all), sums go over distributed shared memory, one cluster barrier each.  The
// draw finds the warp's piece from the sums, its CTA splits that piece over its
// warps again, and the one that holds the token goes through its share in order.
//
// What bounds it.  One chain of 7 over 32,000 tokens takes 6.5 us: dependent loads
// (rows, tokens, entries, the row, its piece again) and two cluster barriers.  64
// chains over 131,072 take 19.5 us: 67 MB at half the copy rate, behind and before
// the same chain.  12 trees of 15 to 63 over 100,003 tokens: 31 us, two to five
// rounds each of some 5 us, a barrier and a reduction in each.
#include <cooperative_groups.h>

#include "ctx_kv_device.cuh"
#include "ctx_kv_internal.h"
#include "draft_step_internal.h"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kMost = 16;
constexpr int kStep = 128;  // entries that a warp takes at once
// Entries of p and q that a warp of a tree's CTA can keep in shared memory: two CTAs fit an SM.
// 12 trees of 15 to 63 over 100,003 tokens 31.4 us, 35.7 with their rows read again in every
// round; 8 over 131,072 27.6 and 29.9.  Larger pieces are read again: 12 over 131,072 31.5 us,
// 20 41, 150 over 32,000 47.
constexpr int kKept = 512;
constexpr double kUnit = 70368744177664.0;  // 2^46

typedef unsigned long long u64;

__device__ __forceinline__ float clean(float x) { return __saturatef(x); }  // to [0, 1]; NaN: 0

// x in [0, 1] as two integers, hi of 2^-23 and, of what that leaves, lo of 2^-46
// to nearest even, offset by kHi and kLo: sums and differences are taken of the
// offset ones.
constexpr int kHi = 0x4b000000, kLo = 0x4b400000;

__device__ __forceinline__ void split(float x, int &hi, int &lo)
{
    constexpr float k = 8388608.0f;  // 2^23
    const float t = fmaf(x, k, k);                   // bits: kHi + the nearest integer to x 2^23
    const float rest = fmaf(x, k, __fsub_rn(k, t));  // exact, at most 1/2
    hi = __float_as_int(t);
    lo = __float_as_int(fmaf(rest, k, 1.5f * k));    // bits: kLo + the nearest integer to rest 2^23
}

__device__ __forceinline__ int64_t joined(int hi, int lo) { return (int64_t)hi * 8388608 + lo; }

// x in [0, 1] in units of 2^-46
__device__ __forceinline__ int64_t fixed(float x)
{
    int hi, lo;
    split(x, hi, lo);
    return joined(hi - kHi, lo - kLo);
}

template <bool BF16>
__device__ __forceinline__ const unsigned char *row_of(const void *base, int64_t stride, int64_t row)
{
    return static_cast<const unsigned char *>(base) + row * stride * (BF16 ? 2 : 4);
}

template <bool BF16>
__device__ __forceinline__ float entry(const unsigned char *row, int64_t i)
{
    if (BF16)
        return clean(__uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + i) << 16));
    return clean(__ldg(reinterpret_cast<const float *>(row) + i));
}

// Entries i .. i + 3 as they are; those from n on 0.  wide: the row takes loads of four.
template <bool BF16>
__device__ __forceinline__ void load4(const unsigned char *row, int64_t i, int64_t n, bool wide, float (&x)[4])
{
    if (wide && i + 4 <= n) {
        if constexpr (BF16) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + i * 2));
            x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
            x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(row + i * 4));
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        x[k] = 0.0f;
        if (i + k < n) {
            if constexpr (BF16)
                x[k] = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + i + k) << 16);
            else
                x[k] = __ldg(reinterpret_cast<const float *>(row) + i + k);
        }
    }
}

// S, and as a sum of two fp32 numbers (48 bits).
struct Share {
    double s;
    float hi, lo;
    __device__ __forceinline__ void set(double x)
    {
        s = x;
        hi = (float)x;
        lo = (float)(x - (double)hi);
    }
};

enum Left { kAll, kLessQ, kLessSQ };  // R = p; max(p - q, 0); max(p - S q, 0)

// Adds one entry of what is left to (hi, lo), units of 2^-23 and 2^-46.
template <int LEFT>
__device__ __forceinline__ void add_left(float p, float q, const Share &s, int &hi, int &lo)
{
    int xh, xl, yh = kHi, yl = kLo;
    const float x = clean(p);
    split(x, xh, xl);
    if constexpr (LEFT == kAll) {
        hi += xh - yh, lo += xl - yl;
    } else if constexpr (LEFT == kLessQ) {
        const float y = clean(q);
        split(y, yh, yl);
        if (x > y)
            hi += xh - yh, lo += xl - yl;
    } else {
        // S q as y + rest; a y above 1 leaves nothing.  rest0 is up to one and a half steps of
        // y0: with y0 from 1/2 on more than r can count, with y0 of 2^-24 to 2^-23, whose steps
        // are half units, enough to take a unit from a p that rounds to the same whole one.
        // Summed once more (exactly: |rest0| < y0), rest is at most half a step of y: r counts
        // it, it rounds to 0 below 2^-23, and an entry is never below 0.
        const float z = clean(q), y0 = __fmul_rn(z, s.hi), rest0 = fmaf(z, s.lo, fmaf(z, s.hi, -y0));
        const float y = __fadd_rn(y0, rest0), rest = __fsub_rn(rest0, __fsub_rn(y, y0));
        split(y, yh, yl);
        const int r = __float_as_int(fmaf(rest, 70368744177664.0f, 12582912.0f)) - kLo;  // rest 2^46 to the nearest integer
        if (y <= 1.0f && __fsub_rn(x, y) > rest)
            hi += xh - yh, lo += xl - yl - r;
    }
}

__device__ __forceinline__ u64 warp_sum(u64 x)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// N entries of what is left, in 32 bits until they are joined
template <int LEFT, int N>
__device__ __forceinline__ u64 left_of(const float (&p)[N], const float (&q)[N], const Share &s)
{
    static_assert(N <= 64, "32-bit sums");
    int hi = 0, lo = 0;
#pragma unroll
    for (int k = 0; k < N; k++)
        add_left<LEFT>(p[k], q[k], s, hi, lo);
    return (u64)joined(hi, lo);
}

template <int LEFT>
__device__ __forceinline__ u64 left_of_one(float p, float q, const Share &s)
{
    int hi = 0, lo = 0;
    add_left<LEFT>(p, q, s, hi, lo);
    return (u64)joined(hi, lo);
}

template <bool TB, int DK>  // target bf16; draft: 0 none, 1 fp32, 2 bf16
struct Rows {
    const unsigned char *p, *q;
    bool wide;

    __device__ __forceinline__ Rows(const VerifyParams &a, int64_t row)
    {
        p = row_of<TB>(a.target, a.target_stride, row);
        q = DK ? row_of<DK == 2>(a.draft, a.draft_stride, row) : p;
        wide = (((uintptr_t)p & (TB ? 7 : 15)) | ((uintptr_t)q & (DK == 0 ? (TB ? 7 : 15) : DK == 2 ? 7 : 15))) == 0;
    }
};

// This lane's entries of a warp's piece [from, to) of a row.  (Functions of their
// own: inlined where they are used, the kernel was four times as long, and half of
// a short launch went into fetching it.)
template <bool TB, int DK, int LEFT>
__device__ __noinline__ u64 sum_of(Rows<TB, DK> rows, int64_t from, int64_t to, Share s)
{
    const int lane = threadIdx.x & 31;
    u64 t = 0;
    constexpr int kU = 4;
    int64_t i = from + 4 * lane;
    for (; i - 4 * lane + kU * kStep <= to; i += kU * kStep) {
        float x[kU][4], y[kU][4];
#pragma unroll
        for (int u = 0; u < kU; u++) {
            load4<TB>(rows.p, i + u * kStep, to, rows.wide, x[u]);
            if (LEFT != kAll)
                load4<DK == 2>(rows.q, i + u * kStep, to, rows.wide, y[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; u++)
            t += left_of<LEFT>(x[u], LEFT != kAll ? y[u] : x[u], s);
    }
    for (; i < to; i += kStep) {
        float x[4], y[4];
        load4<TB>(rows.p, i, to, rows.wide, x);
        if (LEFT != kAll)
            load4<DK == 2>(rows.q, i, to, rows.wide, y);
        t += left_of<LEFT>(x, LEFT != kAll ? y : x, s);
    }
    return t;
}

template <bool TB, int DK>
__device__ __forceinline__ u64 sum_of(const Rows<TB, DK> &rows, Left kind, int64_t from, int64_t to, const Share &s)
{
    if (DK == 0 || kind == kAll)
        return sum_of<TB, DK, kAll>(rows, from, to, s);
    return kind == kLessQ ? sum_of<TB, DK, kLessQ>(rows, from, to, s) : sum_of<TB, DK, kLessSQ>(rows, from, to, s);
}

// The same of a piece of up to kKept entries that is kept in shared memory:
// loaded where `fresh`, read from there in the next rounds of the same row.
template <bool TB, int DK>
__device__ __noinline__ u64 sum_of_kept(Rows<TB, DK> rows, Left kind, int64_t from, int64_t to, Share s, float4 *kept, bool fresh)
{
    const int lane = threadIdx.x & 31;
    constexpr int kU = kKept / kStep;
    float x[kU][4], y[kU][4];
    if (fresh) {
#pragma unroll
        for (int u = 0; u < kU; u++) {
            const int64_t i = from + u * kStep + 4 * lane;
            load4<TB>(rows.p, i, to, rows.wide, x[u]);
            load4<DK == 2>(rows.q, i, to, rows.wide, y[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; u++) {
            kept[(2 * u) * 32 + lane] = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
            kept[(2 * u + 1) * 32 + lane] = make_float4(y[u][0], y[u][1], y[u][2], y[u][3]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kU; u++) {
            *reinterpret_cast<float4 *>(x[u]) = kept[(2 * u) * 32 + lane];
            *reinterpret_cast<float4 *>(y[u]) = kept[(2 * u + 1) * 32 + lane];
        }
    }
    u64 t = 0;
#pragma unroll
    for (int u = 0; u < kU; u++)
        t += kind == kAll ? left_of<kAll>(x[u], x[u], s) : kind == kLessQ ? left_of<kLessQ>(x[u], y[u], s) : left_of<kLessSQ>(x[u], y[u], s);
    return t;
}

// What warp 0 of a tree's CTA tells the others.
struct Step {
    int cur, count, lost;  // row reached, tokens accepted, entries of `gone`
    Left kind;
    float hi, lo;          // S
    bool done;
};

template <bool TB, int DK>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams a)
{
    __shared__ float tp[kVerifyRows], tq[kVerifyRows], tu[kVerifyRows];  // the rows' entries and random numbers
    __shared__ int token[kVerifyRows];                                   // -1: out of range
    __shared__ int16_t parent[kVerifyRows], path[kVerifyRows];
    __shared__ int gone[kVerifyRows];                                    // rejected tokens of the last row (no draft)
    __shared__ u64 sums[2][kMost], pieces[kWarps], parts[kWarps];
    __shared__ int first_lost;
    __shared__ Step walk;
    extern __shared__ float4 kept[];  // trees, pieces of up to kKept entries: [warps][kKept / kStep][p, q][32]
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // waited for where the first sum is exchanged
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), b = blockIdx.x / nc;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned flags = 0;

    const int r0 = __ldg(a.row_start + b), r1 = __ldg(a.row_start + b + 1);
    int n = r1 - r0;
    if (r0 < 0 || r1 < r0 || r1 > a.num_rows || n > kVerifyRows) {
        flags |= kFlagLength;
        n = 0;
    }
    int64_t *out_tokens = a.out_tokens + (int64_t)b * (a.max_accepted + 1);
    int32_t *out_rows = a.out_rows + (int64_t)b * a.max_accepted;

    // ---- the rows: all their loads at once
    for (int i = tid; i < n; i += kThreads) {
        int up = i - 1;
        int64_t x = -1;
        if (i > 0) {
            x = __ldg(a.tokens + r0 + i);
            if (a.parents)
                up = __ldg(a.parents + r0 + i);
            if (up < 0 || up >= i) {
                up = -1;
                flags |= kFlagRow;
            }
            if (x < 0 || x >= a.vocab) {
                x = -1;
                flags |= kFlagRow;
            }
        }
        const bool there = up >= 0 && x >= 0;
        parent[i] = (int16_t)up;
        token[i] = (int)x;
        tp[i] = there ? entry<TB>(row_of<TB>(a.target, a.target_stride, r0 + up), x) : 0.0f;
        if (DK)
            tq[i] = there ? entry<DK == 2>(row_of<DK == 2>(a.draft, a.draft_stride, r0 + up), x) : 0.0f;
        tu[i] = clean(__ldg(a.uniforms + r0 + i));
    }
    if (tid == 0)
        first_lost = kVerifyRows;
    __syncthreads();

    // pieces of the vocabulary: warp g of the cluster has [g * piece, (g + 1) * piece)
    const int64_t all = (int64_t)nc * kWarps, piece = (a.vocab + all * kStep - 1) / (all * kStep) * kStep;
    const bool keep = DK != 0 && a.parents && piece <= kKept;
    int round = 0, lost = 0, kept_row = -1;  // lost: entries of `gone`; kept_row: the row in `kept`
    Share share;
    share.set(1.0);
    share.s = 0.0;
    // sum of what is left of row `cur`: pieces[] holds this CTA's warps', sums[] the CTAs'
    auto total = [&](int cur, Left kind) -> u64 {
        const Rows<TB, DK> rows(a, r0 + cur);
        const int64_t g = (int64_t)rank * kWarps + warp;
        u64 t;
        if (keep) {
            t = sum_of_kept(rows, kind, g * piece, min((g + 1) * piece, a.vocab), share, kept + warp * (kKept / 2), cur != kept_row);
            kept_row = cur;
        } else {
            t = sum_of(rows, kind, g * piece, min((g + 1) * piece, a.vocab), share);
        }
        t = warp_sum(t);
        if (DK == 0)
            for (int k = 0; k < lost; k++)
                if (gone[k] / piece == g)
                    t -= (u64)fixed(entry<TB>(rows.p, gone[k]));
        if (lane == 0)
            pieces[warp] = t;
        __syncthreads();
        u64 c = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++)
            c += pieces[w];
        if (round == 0)  // every CTA of the cluster runs: its shared memory may be written
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < nc)
            cluster.map_shared_rank(&sums[round & 1][0], tid)[rank] = c;
        cluster.sync();
        c = 0;
        for (int r = 0; r < nc; r++)
            c += sums[round & 1][r];
        round++;
        return c;
    };

    // ---- the walk
    int cur = 0, count = 0;
    Left kind = kAll;  // what the rejections behind the last row leave
    const int limit = min(n - 1, a.max_accepted);
    if (!a.parents) {
        for (int i = 1 + tid; i <= limit; i += kThreads) {
            const bool take = DK ? (double)tu[i] * tq[i] < (double)tp[i] : tu[i] < tp[i];
            if (!take)
                atomicMin(&first_lost, i);
        }
        __syncthreads();
        if (n > 0) {
            count = min(first_lost - 1, limit);
            cur = count;
            if (count < limit) {
                if (DK == 0) {
                    if (token[cur + 1] >= 0) {
                        if (tid == 0)
                            gone[0] = token[cur + 1];
                        lost = 1;
                    }
                } else {
                    kind = kLessQ;
                }
            }
            for (int i = tid; i < count; i += kThreads)
                path[i] = (int16_t)(i + 1);
        }
    } else if (n > 0) {
        // Warp 0 walks, and hands the row and S over where it needs the sum of what
        // is left.  (64-bit floating point runs at a fraction of the rate: walked by
        // all warps alike, a batch of trees took 61 us, not 31.)
        int last = 0, lost_now = 0;  // the child tested last; entries of `gone`
        double z = 1.0, q_gone = 0.0;
        bool stale = false;          // z is of the round before
        for (;;) {
            if (warp == 0) {
                bool done = false;
                while (!done) {
                    // the next child in row order
                    int child = 0;
                    if (count < a.max_accepted)
                        for (int i0 = last + 1; i0 < n && child == 0; i0 += 32) {
                            const unsigned hit = __ballot_sync(0xffffffffu, i0 + lane < n && parent[i0 + lane] == cur);
                            if (hit)
                                child = i0 + __ffs(hit) - 1;
                        }
                    if (child == 0) {
                        done = true;
                        break;
                    }
                    if (stale)
                        break;  // for its test the sum is needed
                    const double p = tp[child], u = tu[child];
                    bool take;
                    if (DK) {
                        const double q = tq[child], left = a.replacement ? 1.0 : 1.0 - q_gone;
                        if (!(left > 0x1p-24) || !(z > 0.0)) {
                            done = true;
                            break;
                        }
                        take = u * (q / left) * z < fmax(p - share.s * q, 0.0);
                        if (!take) {
                            share.set(share.s + z / left);
                            q_gone += q;
                            stale = true;
                        }
                    } else {
                        bool before = token[child] < 0;
                        for (int k = 0; k < lost_now; k++)
                            before |= gone[k] == token[child];
                        const double r = before ? 0.0 : p;
                        if (!(z > 0.0)) {
                            done = true;
                            break;
                        }
                        take = u * z < r;
                        if (!take) {
                            z -= r;
                            if (!before) {
                                __syncwarp();
                                if (lane == 0)
                                    gone[lost_now] = token[child];
                                __syncwarp();
                                lost_now++;
                            }
                        }
                    }
                    last = child;
                    if (take) {
                        if (lane == 0)
                            path[count] = (int16_t)child;
                        count++;
                        cur = child;
                        share.s = 0.0, z = 1.0, q_gone = 0.0;
                        stale = false;
                        lost_now = 0;
                    }
                }
                if (lane == 0)
                    walk = Step{cur, count, lost_now, share.s == 0.0 ? kAll : share.s == 1.0 ? kLessQ : kLessSQ, share.hi, share.lo, done};
            }
            __syncthreads();
            const Step w = walk;
            cur = w.cur, count = w.count, lost = w.lost, kind = w.kind;
            share.hi = w.hi, share.lo = w.lo;
            if (w.done)
                break;
            const u64 mass = total(cur, kind);
            if (warp == 0) {
                z = (double)mass / kUnit;
                stale = false;
            }
        }
    }
    __syncthreads();

    // ---- what is known: written before the barrier that the draw waits at
    if (rank == 0) {
        for (int i = tid; i <= a.max_accepted; i += kThreads) {
            out_tokens[i] = i < count ? (int64_t)token[path[i]] : -1;
            if (i < a.max_accepted)
                out_rows[i] = i < count ? path[i] : -1;
        }
        if (tid == 0)
            a.counts[b] = count;
    }
    if (n > 0) {
        // ---- the last token
        u64 mass = total(cur, kind);
        if (mass == 0 && (kind != kAll || lost)) {  // the rejections left nothing
            kind = kAll;
            lost = 0;
            mass = total(cur, kind);
        }
        if (mass == 0)
            flags |= kFlagRow;
        // t = floor(u mass) < mass
        const uint32_t bits = __float_as_uint(tu[0]), e = max(bits >> 23, 1u);
        const u64 m = bits >> 23 ? (bits & 0x7fffffu) | 0x800000u : bits, hi = __umul64hi(m, mass), lo = m * mass;
        const uint32_t sh = 150 - e;  // 23 .. 149
        u64 t = sh < 64 ? (lo >> sh) | (hi << (64 - sh)) : sh < 128 ? hi >> (sh - 64) : 0;
        t = min(t, mass - 1);  // u of 1
        u64 before = 0, mine = sums[(round - 1) & 1][rank];
        for (int r = 0; r < rank; r++)
            before += sums[(round - 1) & 1][r];
        if (mass != 0 && t >= before && t - before < mine) {
            t -= before;
            int w = 0;
            while (w < kWarps - 1 && t >= pieces[w])
                t -= pieces[w++];
            // the piece, split over the warps again
            const Rows<TB, DK> rows(a, r0 + cur);
            const int64_t from = ((int64_t)rank * kWarps + w) * piece, to = min(from + piece, a.vocab);
            const int64_t part = (piece + kWarps * kStep - 1) / (kWarps * kStep) * kStep;
            const int64_t mine0 = from + warp * part, mine1 = min(mine0 + part, to);
            u64 x = 0;
            if (mine0 < mine1) {
                x = warp_sum(sum_of(rows, kind, mine0, mine1, share));
                if (DK == 0)
                    for (int k = 0; k < lost; k++)
                        if (gone[k] >= mine0 && gone[k] < mine1)
                            x -= (u64)fixed(entry<TB>(rows.p, gone[k]));
            }
            if (lane == 0)
                parts[warp] = x;
            __syncthreads();
            w = 0;
            while (w < kWarps - 1 && t >= parts[w])
                t -= parts[w++];
            if (w == warp) {
                for (int64_t i0 = mine0; i0 < mine1; i0 += kStep) {
                    const int64_t i = i0 + 4 * lane;
                    float p[4], q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    u64 v[4], s = 0;
                    load4<TB>(rows.p, i, mine1, rows.wide, p);
                    if (kind != kAll)
                        load4<DK == 2>(rows.q, i, mine1, rows.wide, q);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        v[k] = kind == kAll ? left_of_one<kAll>(p[k], q[k], share)
                               : kind == kLessQ ? left_of_one<kLessQ>(p[k], q[k], share) : left_of_one<kLessSQ>(p[k], q[k], share);
                        if (DK == 0)
                            for (int g = 0; g < lost; g++)
                                if (gone[g] == i + k)
                                    v[k] = 0;
                        s += v[k];
                    }
                    u64 up = s;  // with the lanes before
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const u64 y = __shfl_up_sync(0xffffffffu, up, d);
                        if (lane >= d)
                            up += y;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, up > t);
                    if (hit) {
                        if (lane == __ffs(hit) - 1) {
                            u64 c = up - s;
                            int k = 0;
                            while (k < 3 && c + v[k] <= t)
                                c += v[k++];
                            out_tokens[count] = i + k;
                        }
                        break;
                    }
                    t -= __shfl_sync(0xffffffffu, up, 31);
                }
            }
        }
    }
    if (round == 0)  // (a request without rows)
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && a.error_flags)
        atomicOr(a.error_flags, flags);
}

template <bool TB, int DK>
cudaError_t launch(const VerifyParams &p, int nc, cudaStream_t stream)
{
    // (driver calls that cost nothing next to the launch; no state to keep per device)
    const int64_t all = (int64_t)nc * kWarps, piece = (p.vocab + all * kStep - 1) / (all * kStep) * kStep;
    const int smem = DK != 0 && p.parents && piece <= kKept ? kWarps * kKept * 8 : 0;
    cudaError_t e = nc > 8 ? cudaFuncSetAttribute(verify_kernel<TB, DK>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
    if (e == cudaSuccess && smem > 0)
        e = cudaFuncSetAttribute(verify_kernel<TB, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl_grid(verify_kernel<TB, DK>, dim3((unsigned)p.num_requests * nc), kThreads, smem, nc, stream, p);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    // CTAs of a request: two per SM over all requests, each with some work
    int nc = 1;
    while (nc < kMost && (int64_t)p.num_requests * nc <= sms && p.vocab > (int64_t)2048 * nc)
        nc *= 2;
    if (!p.draft)
        return p.target_bf16 ? launch<true, 0>(p, nc, stream) : launch<false, 0>(p, nc, stream);
    if (p.draft_bf16)
        return p.target_bf16 ? launch<true, 2>(p, nc, stream) : launch<false, 2>(p, nc, stream);
    return p.target_bf16 ? launch<true, 1>(p, nc, stream) : launch<false, 1>(p, nc, stream);
}

}  // namespace dspark
