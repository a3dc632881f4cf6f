// New tokens' K and V into a page-scaled cache (sm_103a).
//
// Mathematics.  For a page and head, K and V apart: e = the least with max |x| <=
// 448 * 2^e over the finite new x, kept to [-32, 31] and to the page's scale where
// it holds context tokens; codes are e4m3(x * 2^-e).  448 = 1.75 * 2^8, so for
// max |x| = 1.f * 2^E, e = E - 8, or E - 7 where 1.f > 1.75.  x * 2^-e is exact
// in fp32, the code's rounding the only one.  A page whose scale grows has its
// codes divided by a power of two (page_scale.cuh).
//
// Work.  A unit is one (request, page, head, K or V); its tokens are read once: a
// thread keeps up to kHold 16-byte words while the CTA finds the maximum (64
// tokens of D 128; more are read again, from L1).  8,192 tokens of 8 heads take 13.5 us,
// 50 MB at 55% of the copy rate, 7 tokens of 64 requests 6.0 us.  What bounds them: the
// first no unit alone, issue slots 60%, DRAM 27%: of a warp's 11.8 cycles an instruction
// 2.7 go into waiting for loads (a unit's page and tokens are loaded when the one
// before is stored), 2.5 into fixed latencies, 1.5 into waiting for a slot, 1.1 into
// barriers; the second one wave of dependent loads (lengths, page, tokens).  With the words in shared memory twelve CTAs fit an SM, not eight
// (14.3 and 9.7 us); infinities and NaN left out word by word cost 1.3 us.  Lengths
// are on the device, so each CTA sums the requests' units itself and takes an
// equal share of them, as the attention does.  A CTA has 128 threads, so that
// a draft step's units (7 tokens of 256 bytes) are there all at once.
#include <type_traits>

#include "draft_step_internal.h"
#include "page_scale.cuh"
#include "tree_attn_mma.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kHold = 8, kCtas = 8;

struct Fresh {
    int q0, n, ctx;
};

__device__ __forceinline__ Fresh request_of(const InsertScaledParams &p, int b, unsigned &flags)
{
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), ctx = __ldg(p.context_lens + b);
    Fresh r{q0, q1 - q0, ctx};
    if (q0 < 0 || q1 < q0 || q1 > p.num_rows || ctx < 0 ||
        (q1 > q0 && (int64_t)ctx + (q1 - q0) > p.table_blocks * p.block_size)) {
        flags |= kFlagLength;
        r.n = 0;
    }
    return r;
}

__device__ __forceinline__ int pages_of(const Fresh &r, int bs)
{
    return r.n ? (r.ctx + r.n - 1) / bs - r.ctx / bs + 1 : 0;
}

// max of |x| of bf16 pairs, by their bits; FINITE: over the finite ones
template <bool FINITE>
__device__ __forceinline__ uint32_t top2(uint32_t top, uint32_t w)
{
    w &= 0x7fff7fffu;
    if (FINITE)
        w &= ~__vcmpgeu2(w, 0x7f807f80u);
    return __vmaxu2(top, w);
}

template <bool FINITE>
__device__ __forceinline__ uint32_t top8(uint32_t top, const uint4 &v)
{
    return top2<FINITE>(top2<FINITE>(top2<FINITE>(top2<FINITE>(top, v.x), v.y), v.z), v.w);
}

__device__ __forceinline__ int exponent_of(uint32_t bits)  // of the largest |x|, as bf16 bits
{
    const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u);
    return min(max(e, kScaleMin), kScaleMax);
}

// eight values times s as codes
__device__ __forceinline__ uint2 encode8(const uint4 &v, float s)
{
    const uint64_t s2 = pr(s, s);
    return make_uint2(e4m3x4(mul2(bf2_to_f2(v.x), s2), mul2(bf2_to_f2(v.y), s2)),
                      e4m3x4(mul2(bf2_to_f2(v.z), s2), mul2(bf2_to_f2(v.w), s2)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtas) insert_scaled_kernel(const __grid_constant__ InsertScaledParams p)
{
    constexpr int kW = D / 8, kStep = kThreads / kW;  // 16-byte words of a token's K or V; tokens at once
    __shared__ int64_t scratch[kWarps + 4];
    __shared__ uint32_t tops[2][kWarps];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.num_kv_heads, bs = p.block_size;
    unsigned flags = 0;
    const attn::Find f = attn::find_request<kThreads>(
        p.num_requests, scratch, [&](int b) { return (int64_t)pages_of(request_of(p, b, flags), bs) * (2 * H); });
    const attn::Shares shares(f.total, gridDim.x);
    if (f.b >= 0) {
        int b = f.b;
        unsigned ignore = 0;
        Fresh r = request_of(p, b, ignore);
        const int64_t u0 = shares.start(blockIdx.x), u1 = shares.start(blockIdx.x + 1);
        int64_t of = u0 - f.before;  // the unit's number in its request
        int turn = 0;
        const int w = tid % kW;
        for (int64_t u = u0; u < u1; u++, of++) {
            while (of >= (int64_t)pages_of(r, bs) * (2 * H)) {
                of -= (int64_t)pages_of(r, bs) * (2 * H);
                r = request_of(p, ++b, ignore);
            }
            // K and V of a head one after the other: their codes lie side by side
            const int pi = (int)attn::Shares::div(of, 2 * H), hp = (int)(of - (int64_t)pi * (2 * H)), h = hp >> 1, part = hp & 1;
            const int blk = r.ctx / bs + pi;
            const int64_t first = (int64_t)blk * bs;
            const int lo = pi ? (int)first : r.ctx, hi = (int)min((int64_t)r.ctx + r.n, first + bs);
            const int held = pi ? 0 : r.ctx - (int)first;  // the context's tokens in the page
            const int64_t page = __ldg(p.table + b * p.table_stride + blk);
            const uint16_t *src = (part ? p.v + h * p.v_hs : p.k + h * p.k_hs) + w * 8;
            const int64_t ts = part ? p.v_ts : p.k_ts;
            const int row0 = r.q0 + lo - r.ctx, rows = hi - lo;
            uint4 v[kHold];
#pragma unroll
            for (int k = 0; k < kHold; k++)
                if (k * kStep < rows) {  // the same for all
                    const int x = tid / kW + k * kStep;
                    v[k] = x < rows ? __ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts)) : make_uint4(0, 0, 0, 0);
                }
            if (page < 0 || page >= p.num_blocks) {
                flags |= kFlagBlockRange;
                continue;
            }
            const int was = held ? page_exponent(p.scales, page, H, h, part) : kScaleMin;
            // the largest |x| of the CTA's tokens
            auto largest = [&](auto finite) {
                constexpr bool kFinite = decltype(finite)::value;
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < kHold; k++)
                    if (k * kStep < rows)
                        top = top8<kFinite>(top, v[k]);
                for (int x = tid / kW + kHold * kStep; x < rows; x += kStep)
                    top = top8<kFinite>(top, __ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts)));
                top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
                if (lane == 0)
                    tops[turn][warp] = top;
                __syncthreads();  // everyone has read the old scale too
#pragma unroll
                for (int i = 0; i < kWarps; i++)
                    top = max(top, tops[turn][i]);
                turn ^= 1;
                return top;
            };
            uint32_t top = largest(std::false_type{});
            if (top >= 0x7f80u)  // infinities or NaN among them: once more without these
                top = largest(std::true_type{});
            const int e = max(exponent_of(top), was);
            unsigned char *codes = p.cache + ((page * H + h) * bs) * (int64_t)(2 * D) + part * D;
            // the codes of the context's tokens in the page, where the scale grows
            if (held && e > was)
                for (int x = tid; x < held * (D / 16); x += kThreads) {
                    uint4 *at = reinterpret_cast<uint4 *>(codes + (int64_t)(x / (D / 16)) * (2 * D) + x % (D / 16) * 16);
                    *at = scale_codes(*at, half2_power(e - was));
                }
            if (tid == 0)
                p.scales[(page * H + h) * 2 + part] = (int8_t)e;
            const float s = __int_as_float((127 - e) << 23);
            unsigned char *dst = codes + (int64_t)(lo - first) * (2 * D) + w * 8;
#pragma unroll
            for (int k = 0; k < kHold; k++)
                if (k * kStep < rows) {
                    const int x = tid / kW + k * kStep;
                    if (x < rows)
                        *reinterpret_cast<uint2 *>(dst + (int64_t)x * (2 * D)) = encode8(v[k], s);
                }
            for (int x = tid / kW + kHold * kStep; x < rows; x += kStep)
                *reinterpret_cast<uint2 *>(dst + (int64_t)x * (2 * D)) =
                    encode8(__ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts)), s);
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

}  // namespace

cudaError_t launch_insert_scaled(const InsertScaledParams &p, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int64_t units = p.num_rows * p.num_kv_heads * 2;  // at most: a page each
    const int ctas = (int)(units < kCtas * (int64_t)sms ? units : kCtas * (int64_t)sms);
    switch (p.head_dim) {
    case 64: return launch_pdl(insert_scaled_kernel<64>, ctas, kThreads, 0, stream, p);
    case 128: return launch_pdl(insert_scaled_kernel<128>, ctas, kThreads, 0, stream, p);
    default: return launch_pdl(insert_scaled_kernel<256>, ctas, kThreads, 0, stream, p);
    }
}

}  // namespace dspark
