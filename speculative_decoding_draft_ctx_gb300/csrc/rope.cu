// sm_103a kernels of the cos|sin table and of rotary positions with the K/V
// insert.
//
// Defining passages: DSpark context-KV writer page, module docstring (partial
// NeoX RoPE from a cos|sin cache, the cache layout, fp8 of x / scale, slots
// < 0 not written); DSpark draft model page (the cos_sin_cache whose last dim
// is rotary_dim).  The interleaved pairing and the scaled frequencies are the
// usual forms those pages do not use.
//
// Table.  The angle p f of a far position in fp32 loses the turn it is in.
// Here the frequency is a 64-bit fixed-point fraction F = f / 2 pi * 2^64 of a
// turn, so p F mod 2^64 is the angle's fraction of a turn, exact but for F's
// own rounding (p 2^-64 turns, 2^-30 radians at position 2^31): the wrap of
// the integer product is the range reduction.  The top bits give the nearest quarter turn, the signed rest
// x (|x| <= pi/4) goes to fp32 with a relative rounding and into the Taylor
// series of sine (to x^9: the next term is below 2^-28.7 x) and cosine (to
// x^8: below 2^-25); with the roundings of fp32 an entry is off by 2^-22 at
// most.  A thread makes 4 neighbouring angles, so it stores 8 or 16
// bytes of cos and of sin, and stays with them from row to row: the next
// angle is a 64-bit sum.  Bound: some 40 instructions per angle (131,072
// positions of 64 entries: 9.1 us, the bytes' time 2.5; the instructions alone
// would take half of that).
//
// Rotation.  A head row of D dims is held by D / 8 lanes, 8 dims (16 bytes)
// each, so a warp takes 256 / D rows at once.  Half layout: the partner of
// dim i < r/2 is i + r/2, r/16 lanes away: one shuffle per word.
// Interleaved: both dims of a pair are in one lane.  Where a row is not
// 16-byte aligned, or r/2 is no whole number of lanes, the same code loads
// its elements and partners one by one (before any store of the warp, so in
// place is safe).  Per element the arithmetic is x1 c - x2 s in fp32 (the
// product of two bf16 values is exact there), rounded once to bf16.  Bound:
// the read and write of q and k.  A warp's unit is kBatch row groups of one
// token: their loads go out before the position is waited for and the cos|sin
// words (whole 8- or 16-byte loads) after it, so a unit waits twice; four
// CTAs per SM keep 32 warps' units in flight (with a CTA per token, 104
// registers and a scalar load per cos and sin, a prefill batch of 8,192 tokens into an fp8
// cache took 97 us; it takes 46, the bytes' time 30).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ctx_kv_device.cuh"
#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace dspark {
namespace {

// ------------------------------------------------------------------ the table

constexpr int kTableThreads = 256;

// cos and sin of 2 pi u 2^-64
__device__ __forceinline__ void turn_cos_sin(uint64_t u, float &c, float &s)
{
    const uint64_t quarter = (u + (1ull << 61)) >> 62;  // nearest quarter turn, 0..3 (4 wraps to 0)
    const int64_t rest = (int64_t)(u - (quarter << 62));  // in [-2^61, 2^61)
    const float x = (float)rest * 3.40612158e-19f;  // 2 pi 2^-64: radians, at most pi/4
    const float x2 = x * x;
    const float sn = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f), x);
    const float cs = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 40320.0f, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
    const int n = (int)quarter & 3;
    const float a = (n & 1) ? sn : cs, b = (n & 1) ? cs : sn;
    c = (n == 1 || n == 2) ? -a : a;
    s = (n >= 2) ? -b : b;
}

// V entries per thread: 4 where r/2 is a multiple of 4 (whole 8- or 16-byte
// stores), else 1.
template <bool FP32, int V>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    pdl_enter();
    const int half = p.rotary_dim >> 1, per_row = half / V;
    const unsigned t = blockIdx.x * kTableThreads + threadIdx.x;
    const int step = (int)(gridDim.x * kTableThreads / (unsigned)per_row);  // rows all threads make at once
    const int row0 = (int)(t / (unsigned)per_row), i0 = (int)(t - (unsigned)row0 * per_row) * V;
    if (row0 >= step)
        return;
    uint64_t turn[V], more[V];  // the angles of a row, and from one row to the next
#pragma unroll
    for (int j = 0; j < V; j++) {
        turn[j] = (uint64_t)(p.first + row0) * p.turns[i0 + j];
        more[j] = (uint64_t)step * p.turns[i0 + j];
    }
    for (int64_t row = row0; row < p.count; row += step) {
        float c[V], s[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            turn_cos_sin(turn[j], c[j], s[j]);
            turn[j] += more[j];
            c[j] *= p.amplitude;
            s[j] *= p.amplitude;
        }
        const int64_t at = row * p.rotary_dim + i0;
        if constexpr (FP32) {
            float *o = static_cast<float *>(p.out) + at;
            if constexpr (V == 4) {
                *reinterpret_cast<float4 *>(o) = make_float4(c[0], c[1], c[2], c[3]);
                *reinterpret_cast<float4 *>(o + half) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                o[0] = c[0];
                o[half] = s[0];
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(p.out) + at;
            if constexpr (V == 4) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
                *reinterpret_cast<uint2 *>(o + half) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
            } else {
                o[0] = (uint16_t)pack_bf16x2(c[0], 0.0f);
                o[half] = (uint16_t)pack_bf16x2(s[0], 0.0f);
            }
        }
    }
}

// ------------------------------------------------------------------ the rotation

constexpr int kThreads = 256, kWarps = kThreads / 32, kBatch = 4;
constexpr unsigned kFlagSlot = 0x1u, kFlagPos = 0x2u;

__device__ __forceinline__ float bfl(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bfh(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// eight bf16 values from an address of any 2-byte alignment
__device__ __forceinline__ uint4 gather8(const uint16_t *p)
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        w[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 4 table entries from entry `at` (a multiple of 4; rows start at multiples of 8 entries)
template <bool TF32>
__device__ __forceinline__ void table4(const void *table, int64_t at, float (&o)[4])
{
    if constexpr (TF32) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(table) + at));
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(table) + at));
        o[0] = bfl(v.x), o[1] = bfh(v.x), o[2] = bfl(v.y), o[3] = bfh(v.y);
    }
}

template <bool TF32>
__device__ __forceinline__ float table1(const void *table, int64_t at)
{
    if constexpr (TF32)
        return __ldg(static_cast<const float *>(table) + at);
    else
        return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(table) + at) << 16);
}

// VEC: rows are 16-byte aligned and a lane's 8 dims rotate together (half
// layout: r % 16 == 0; interleaved: r % 8 == 0).
template <int D, bool VEC, bool TF32>
__global__ void __launch_bounds__(kThreads, VEC ? 4 : 2) rope_insert_kernel(const __grid_constant__ RopeInsertParams p)
{
    constexpr int L = D / 8, RPW = 32 / L;  // lanes per row, rows per warp and step
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = lane % L, sub = lane / L;
    const int r = p.rotary_dim, half = r >> 1;
    const int Hq = p.num_heads, Hkv = p.num_kv_heads;
    const bool insert = p.slot_mapping != nullptr;
    const int rows = Hq + Hkv + (insert ? Hkv : 0);  // head rows of a token: q, k and (insert) v
    const int groups = (rows + RPW * kBatch - 1) / (RPW * kBatch);
    const int d0 = 8 * q;                            // the lane's first dim
    const bool turns = d0 < r;                       // VEC: all of its dims turn, or none
    const int lanes_half = r >> 4;                   // VEC, half layout: lanes of one half
    const int partner_lane = q < lanes_half ? lane + lanes_half : q < 2 * lanes_half ? lane - lanes_half : lane;
    const float sign = p.inverse ? -1.0f : 1.0f;
    Fp8Scale ks{}, vs{};
    if (insert && p.fp8) {
        ks = fp8_scale(p.k_scale ? __ldg(p.k_scale) : 1.0f);
        vs = fp8_scale(p.v_scale ? __ldg(p.v_scale) : 1.0f);
    }
    unsigned flags = 0;

    const int64_t units = p.num_tokens * groups, stride = (int64_t)gridDim.x * kWarps;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += stride) {
        const int64_t t = u <= 0x7fffffff ? (int64_t)((uint32_t)u / (uint32_t)groups) : u / groups;
        const int g = (int)(u - t * groups) * RPW * kBatch + sub;  // the lane's first row
        int64_t pos = __ldg(p.positions + t);
        int64_t slot = insert ? __ldg(p.slot_mapping + t) : -1;
        // units of query rows alone, most of them, take one address and a step
        // (a third of the instructions, which bound a prefill batch, were addresses)
        const bool only_q = VEC && g - sub + RPW * kBatch <= Hq;  // uniform over the warp
        uint4 x[kBatch];
        uint32_t partner[VEC ? 1 : kBatch][4];
        if (only_q) {
            const uint16_t *src = p.q + t * p.q_ts + g * p.q_hs + d0;
#pragma unroll
            for (int b = 0; b < kBatch; b++)
                x[b] = *reinterpret_cast<const uint4 *>(src + b * (RPW * p.q_hs));
        }
#pragma unroll
        for (int b = 0; b < kBatch && !only_q; b++) {
            const int hh = g + b * RPW;
            x[b] = make_uint4(0, 0, 0, 0);
            if (hh < rows) {
                const uint16_t *src = hh < Hq         ? p.q + t * p.q_ts + hh * p.q_hs
                                      : hh < Hq + Hkv ? p.k + t * p.k_ts + (hh - Hq) * p.k_hs
                                                      : p.v + t * p.v_ts + (hh - Hq - Hkv) * p.v_hs;
                if constexpr (VEC) {
                    x[b] = *reinterpret_cast<const uint4 *>(src + d0);
                } else {
                    x[b] = gather8(src + d0);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        uint32_t w = 0;
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int d = d0 + 2 * j + e;
                            int m = p.interleaved ? d ^ 1 : (d < half ? d + half : d - half);
                            m = d < r ? m : d;
                            w |= (uint32_t)src[m] << (16 * e);
                        }
                        partner[b][j] = w;
                    }
                }
            }
        }
        const bool turn = pos >= 0 && pos < p.max_pos;
        if (!turn) {
            flags |= kFlagPos;
            slot = -1;
            pos = 0;
        }
        if (slot >= p.capacity) {
            flags |= kFlagSlot;
            slot = -1;
        }
        // cos and signed sin of the lane's dims: out = x c + partner s
        float c[8], s[8];
        if (VEC && turns && turn) {
            const int64_t row = pos * r;
            if (p.interleaved) {
                float cv[4], sv[4];
                table4<TF32>(p.cos_sin, row + (d0 >> 1), cv);
                table4<TF32>(p.cos_sin, row + half + (d0 >> 1), sv);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    c[2 * e] = c[2 * e + 1] = cv[e];
                    s[2 * e] = -sign * sv[e], s[2 * e + 1] = sign * sv[e];
                }
            } else {
                const int i = d0 < half ? d0 : d0 - half;
                const float sg = d0 < half ? -sign : sign;
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    float cv[4], sv[4];
                    table4<TF32>(p.cos_sin, row + i + e, cv);
                    table4<TF32>(p.cos_sin, row + half + i + e, sv);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        c[e + k] = cv[k], s[e + k] = sg * sv[k];
                }
            }
        } else if (!VEC) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int d = d0 + e;
                c[e] = 1.0f, s[e] = 0.0f;
                if (turn && d < r) {
                    const int i = p.interleaved ? d >> 1 : (d < half ? d : d - half);
                    const bool upper = p.interleaved ? (d & 1) : d >= half;
                    c[e] = table1<TF32>(p.cos_sin, pos * r + i);
                    s[e] = (upper ? sign : -sign) * table1<TF32>(p.cos_sin, pos * r + half + i);
                }
            }
            __syncwarp();  // in place: every partner is read before any row of the unit is written
        }
        const int64_t hstride = (int64_t)p.block_size * (2 * D);
        int64_t row0 = 0;
        if (!only_q && slot >= 0) {
            const int64_t blk = slot <= 0x7fffffff ? (int64_t)((uint32_t)slot / (uint32_t)p.block_size) : slot / p.block_size;
            row0 = (blk * Hkv * p.block_size + (slot - blk * p.block_size)) * (2 * D);
        }
        uint16_t *qdst = p.q_out + t * p.qo_ts + g * p.qo_hs + d0;
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const int hh = g + b * RPW;
            if (g - sub + b * RPW >= rows)
                break;  // uniform over the warp
            const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
            uint32_t y[4], pw[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if constexpr (!VEC)
                    pw[j] = partner[b][j];
                else
                    pw[j] = p.interleaved ? (w[j] >> 16) | (w[j] << 16) : __shfl_sync(0xffffffffu, w[j], partner_lane);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                y[j] = w[j];
                if (turn && d0 + 2 * j < r)
                    y[j] = pack_bf16x2(fmaf(bfl(w[j]), c[2 * j], bfl(pw[j]) * s[2 * j]),
                                       fmaf(bfh(w[j]), c[2 * j + 1], bfh(pw[j]) * s[2 * j + 1]));
            }
            if (only_q) {
                *reinterpret_cast<uint4 *>(qdst + b * (RPW * p.qo_hs)) = make_uint4(y[0], y[1], y[2], y[3]);
                continue;
            }
            if (hh >= rows)
                continue;
            if (hh < Hq + Hkv) {
                uint16_t *dst = hh < Hq ? p.q_out + t * p.qo_ts + hh * p.qo_hs : p.k_out + t * p.ko_ts + (hh - Hq) * p.ko_hs;
                if constexpr (VEC) {
                    *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(y[0], y[1], y[2], y[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        dst[d0 + 2 * j] = (uint16_t)y[j];
                        dst[d0 + 2 * j + 1] = (uint16_t)(y[j] >> 16);
                    }
                }
            }
            if (slot >= 0 && hh >= Hq) {
                const bool is_k = hh < Hq + Hkv;
                const uint4 o = is_k ? make_uint4(y[0], y[1], y[2], y[3]) : x[b];
                const int64_t at = row0 + (is_k ? hh - Hq : hh - Hq - Hkv) * hstride + (is_k ? 0 : D) + d0;
                if (p.fp8) {
                    *reinterpret_cast<uint2 *>(p.cache + at) = quantise8(o, is_k ? ks : vs);
                } else {
                    *reinterpret_cast<uint4 *>(p.cache + 2 * at) = o;
                }
            }
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

int sm_count(cudaError_t &e)
{
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int D>
cudaError_t launch_rope_d(const RopeInsertParams &p, cudaStream_t stream)
{
    cudaError_t e;
    const int sms = sm_count(e);
    if (e != cudaSuccess)
        return e;
    const int rows = p.num_heads + p.num_kv_heads * (p.slot_mapping ? 2 : 1);
    const int per = 256 / D * kBatch;  // rows of a unit
    const int64_t want = (p.num_tokens * ((rows + per - 1) / per) + kWarps - 1) / kWarps, most = (p.vec ? 4 : 2) * (int64_t)sms;
    const int blocks = (int)(want < most ? want : most);
    if (p.vec)
        return launch_pdl(p.table_fp32 ? rope_insert_kernel<D, true, true> : rope_insert_kernel<D, true, false>, blocks,
                          kThreads, 0, stream, p);
    return launch_pdl(p.table_fp32 ? rope_insert_kernel<D, false, true> : rope_insert_kernel<D, false, false>, blocks,
                      kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, bool fp32, cudaStream_t stream)
{
    cudaError_t e;
    const int sms = sm_count(e);
    if (e != cudaSuccess)
        return e;
    const int v = (p.rotary_dim >> 1) % 4 == 0 ? 4 : 1;
    const int64_t units = p.count * ((p.rotary_dim >> 1) / v);
    const int64_t want = (units + kTableThreads - 1) / kTableThreads;
    const int blocks = (int)(want < 8 * sms ? want : 8 * sms);
    if (v == 4)
        return launch_pdl(fp32 ? rope_table_kernel<true, 4> : rope_table_kernel<false, 4>, blocks, kTableThreads, 0,
                          stream, p);
    return launch_pdl(fp32 ? rope_table_kernel<true, 1> : rope_table_kernel<false, 1>, blocks, kTableThreads, 0,
                      stream, p);
}

cudaError_t launch_rope_insert(const RopeInsertParams &p, int head_dim, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return launch_rope_d<64>(p, stream);
    case 128: return launch_rope_d<128>(p, stream);
    case 256: return launch_rope_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dspark
