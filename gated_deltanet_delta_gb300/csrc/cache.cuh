// cache.cuh -- rows into a paged attention cache, quantised on the way, and back out of it.
//
// Both are copies: each value is read once and written once, and the bound is HBM.  A row (one token,
// one head, D values) belongs to a group of D / 8 lanes, eight values per lane: 16-byte accesses on the
// 16-bit side, 8-byte accesses on the 8-bit side.  A CTA takes kTokens consecutive tokens of one head of
// K or of V, so that its accesses to the cache run along the tokens of a page; a group has all its rows'
// loads in flight before the first is used.  Measured, prompts of up to 8192 tokens, 16 heads of 128, 292 MB: write 48 us, 89 %
// of a copy's rate; read 45 us, 96 %.
//
// Quantisation (cache type e4m3): per row, scale = the least power of two s with max |x| <= 448 s, and
// the value e4m3(x / s), to nearest, ties to even.  A power of two, because a floating-point type loses
// nothing by it (its relative step is the same at every scale), x / s and value * s are exact, and the
// dequantised value is itself a bf16 (or binary16) number: reading back rounds nothing.  At the source type's
// largest scale (kTop) rounding up to the value 256 would leave the type (256 kTop is its first power of two past the
// largest number), so there such elements take 240, the value below: within a sixteenth, e4m3's relative error
// elsewhere too.  s is at least 2^-100.  A row of zeros gets scale 1.  Elements that are not finite become e4m3's
// NaN and do not count for the scale.
#pragma once

#include <cuda_fp8.h>

#include "attn_mma.cuh"
#include "common.cuh"
#include "kernel_args.h"

namespace gdn {
namespace cache {

constexpr int kThreads = 256;

// The largest of the values that the LANES lanes of a row hold.
template <int LANES>
__device__ __forceinline__ float row_max(float x, unsigned mask) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(mask, x, o));
    return x;
}

// Two floats of at most 448, or NaN, to two e4m3 values (nearest even), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The eight values of a lane, of a row that LANES lanes hold, to e4m3; the row's scale.
template <int LANES, bool F16>
__device__ __forceinline__ uint2 quantise8(const uint32_t (&w)[4], float& scale) {
    constexpr float kTop = F16 ? 0x1p8f : 0x1p120f;  // the largest scale that the type's finite rows have
    float f[8], mx = 0.f;                            // fmaxf passes over NaN
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = attn::unpack2<F16>(w[j]);
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
        mx = fmaxf(mx, fmaxf(fabsf(p.x), fabsf(p.y)));
    }
    mx = row_max<LANES>(mx, kFullMask);
    // Rows of scale kTop, and rows with infinities, which are not to count.  In a branch: as selects in every row
    // both together took 14 % more time.
    if (mx > 224.f * kTop) {
        mx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (fabsf(f[j]) < INFINITY) mx = fmaxf(mx, fabsf(f[j] = fminf(fmaxf(f[j], -240.f * kTop), 240.f * kTop)));
            else f[j] = __int_as_float(0x7fffffff);
        }
        mx = row_max<LANES>(mx, LANES == 32 ? kFullMask : ((1u << LANES % 32) - 1) << (threadIdx.x & (32 - LANES)));
    }
    // 448 = 1.75 2^8: the exponent is mx's less 8, less 7 where mx's significand is over 1.75
    const uint32_t u = __float_as_uint(mx);
    int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) > 0x600000u ? 7 : 8);
    e = max(e, -100);
    if (mx == 0.f) e = 0;
    scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= inv;
    return make_uint2(to_e4m3x2(f[0], f[1]) | to_e4m3x2(f[2], f[3]) << 16, to_e4m3x2(f[4], f[5]) | to_e4m3x2(f[6], f[7]) << 16);
}

// kv: 0 moves keys, 1 values (blockIdx.z).
template <int D, bool F16, bool F8, int TOKENS>
__global__ void __launch_bounds__(kThreads) attn_cache_write_kernel(const __grid_constant__ CacheMoveArgs a) {
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES, ROWS = (TOKENS + GROUPS - 1) / GROUPS;
    __shared__ long long rows_s[TOKENS];
    const int h = blockIdx.y, kv = blockIdx.z, lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const long long t0 = static_cast<long long>(blockIdx.x) * TOKENS;
    const uint16_t* src = (kv ? a.v_in + t0 * a.v_stride : a.k_in + t0 * a.k_stride) + h * D + lane * 8;
    const long long stride = kv ? a.v_stride : a.k_stride;
    uint4 x[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int k = group + i * GROUPS;
        x[i] = k < TOKENS && t0 + k < a.T ? __ldcs(reinterpret_cast<const uint4*>(src + k * stride)) : make_uint4(0, 0, 0, 0);
    }
    // the cached row of each token (-1: none), once per token: a 64-bit division per row and lane took as long as
    // the copy
    if (threadIdx.x < TOKENS) {
        const long long t = t0 + threadIdx.x, slot = t < a.T ? a.slots[t] : -1;
        long long row = -1;
        if (slot >= 0) {  // a negative slot: the token is not kept
            const long long page = (slot | a.page_size) >> 32 ? slot / a.page_size : static_cast<unsigned>(slot) / static_cast<unsigned>(a.page_size);
            if (page < a.num_pages) row = (page * a.H + h) * a.page_size + (slot - page * a.page_size);
            else atomicOr(a.status, kStatusBadCacheIndex);
        }
        rows_s[threadIdx.x] = row;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float scale = 1.f;
        uint2 q = make_uint2(0, 0);
        if constexpr (F8) q = quantise8<LANES, F16>(w, scale);
        const int k = group + i * GROUPS;
        const long long row = k < TOKENS ? rows_s[k] : -1;
        if (row < 0) continue;
        if constexpr (F8) {
            uint8_t* dst = static_cast<uint8_t*>(kv ? a.vc : a.kc);
            *reinterpret_cast<uint2*>(dst + row * D + lane * 8) = q;
            if (lane == 0) (kv ? a.vs : a.ks)[row] = scale;
        } else {
            uint16_t* dst = static_cast<uint16_t*>(kv ? a.vc : a.kc);
            *reinterpret_cast<uint4*>(dst + row * D + lane * 8) = x[i];
        }
    }
}

template <int D, bool F16, bool F8, int TOKENS>
__global__ void __launch_bounds__(kThreads) attn_cache_read_kernel(const __grid_constant__ CacheMoveArgs a) {
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES, ROWS = (TOKENS + GROUPS - 1) / GROUPS;
    __shared__ long long rows_s[TOKENS];
    const int h = blockIdx.y, kv = blockIdx.z, lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const long long t0 = static_cast<long long>(blockIdx.x) * TOKENS;
    const long long most = static_cast<long long>(a.max_pages) * a.page_size;  // tokens that a page table holds
    if (blockIdx.x == 0 && h == 0 && kv == 0) {  // malformed bounds are reported whether or not a row falls to them
        for (int n = threadIdx.x; n < a.num_seqs; n += kThreads) {
            const long long b = a.cu[n], e = a.cu[n + 1];
            if (b < 0 || e < b || e > a.T || e - b > most) atomicOr(a.status, kStatusBadSeqlens);
        }
    }
    if (threadIdx.x < TOKENS) {  // the cached row of each token (-1: none)
        const long long t = t0 + threadIdx.x;
        long long row = -1;
        if (t < a.T) {
            // the last sequence that begins at or before t
            int lo = 0, hi = a.num_seqs;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const long long b = a.cu[lo], e = a.cu[lo + 1], pos = t - b;
            if (b >= 0 && t < e && e <= a.T && pos >= 0 && e - b <= most) {
                const long long pg = pos / a.page_size;
                const long long page = a.table[static_cast<long long>(lo) * a.max_pages + pg];
                if (page >= 0 && page < a.num_pages) row = (page * a.H + h) * a.page_size + (pos - pg * a.page_size);
                else atomicOr(a.status, kStatusBadCacheIndex);
            }
        }
        rows_s[threadIdx.x] = row;
    }
    __syncthreads();
    long long row[ROWS];
    uint4 x[ROWS];
    float s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int k = group + i * GROUPS;
        row[i] = k < TOKENS ? rows_s[k] : -1;
        if constexpr (F8) {
            const uint8_t* src = static_cast<const uint8_t*>(kv ? a.vc : a.kc);
            const uint2 w = row[i] >= 0 ? __ldcs(reinterpret_cast<const uint2*>(src + row[i] * D + lane * 8)) : make_uint2(0, 0);
            x[i] = make_uint4(w.x, w.y, 0, 0);
            s[i] = row[i] >= 0 ? (kv ? a.vs : a.ks)[row[i]] : 0.f;
        } else {
            const uint16_t* src = static_cast<const uint16_t*>(kv ? a.vc : a.kc);
            x[i] = row[i] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(src + row[i] * D + lane * 8)) : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (row[i] < 0) continue;  // nothing cached for this token: its row is not written
        if constexpr (F8) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = (j < 2 ? x[i].x : x[i].y) >> (16 * (j & 1)) & 0xffffu;
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
                const float2 f = __half22float2(__half2(hr));
                w[j] = attn::pack2<F16>(f.x * s[i], f.y * s[i]);
            }
            x[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        uint16_t* dst = kv ? a.v_out : a.k_out;
        __stcs(reinterpret_cast<uint4*>(dst + ((t0 + group + i * GROUPS) * a.H + h) * D + lane * 8), x[i]);
    }
}

// Rotation by position on the way: query rows to q_out, key rows to the cache, and value rows, which are not turned.  The
// pairs (a, b) of features become (a cos - b sin, b cos + a sin), each product and sum rounded to fp32 by itself, so
// that the result does not depend on how a compiler contracts them; the turned row is rounded to its type before it is quantised,
// so that an 8-bit cache holds what attn_cache_write would make of the 16-bit rows.
//
// A copy too: each row is read once and written once.  A group of D / 8 lanes takes up to HEADS heads of one token, all queries, keys or
// values, so that the token's row of the table, its slot and its addresses are there once for HEADS rows; the rows' loads are in
// flight together.  HALVES: feature i's partner is i + turned / 2, in another lane of the group: it comes by a shuffle of the
// packed row.  Else 2 i and 2 i + 1 are partners.
// Measured, prompts of up to 8192 tokens, 32 query and 8 key heads of 128, e4m3: 89 us, 91 % of a copy's rate; of up to 4095 tokens,
// 16 and 4 heads of 256, 16 bits: 88 us, 98 % (with queries, keys and values in one CTA, four heads a group: 106 and 90 us).
template <int D, bool F16, bool F8, bool HALVES, int HEADS>
__global__ void __launch_bounds__(kThreads) attn_cache_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    // a token's heads in consecutive CTAs: those that quantise among those that copy, and the table's rows in L2
    const int qparts = (a.Hq + HEADS - 1) / HEADS, kparts = (a.H + HEADS - 1) / HEADS, parts = qparts + 2 * kparts;
    const int part = blockIdx.x % parts, kind = part < qparts ? 0 : part < qparts + kparts ? 1 : 2;  // queries, keys, values
    const long long t = static_cast<long long>(blockIdx.x / parts) * GROUPS + group;
    const int h0 = (part - (kind > 0 ? qparts : 0) - (kind > 1 ? kparts : 0)) * HEADS, heads = min(HEADS, (kind ? a.H : a.Hq) - h0);
    const bool here = t < a.T;
    const uint16_t* src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h0 * D + lane * 8;
    uint4 x[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) x[i] = here && i < heads ? __ldcs(reinterpret_cast<const uint4*>(src + i * D)) : make_uint4(0, 0, 0, 0);
    const long long pos = here ? a.positions[t] : -1;
    const bool known = pos >= 0 && pos < a.max_pos;
    if (here && !known && lane == 0 && part == 0) atomicOr(a.status, kStatusBadPosition);
    long long row0 = -1;  // the cached row of the first of these heads (-1: none); a negative slot: the token is not kept
    if (known && kind) {
        const long long slot = a.slots[t];
        if (slot >= 0) {
            const long long page = (slot | a.page_size) >> 32 ? slot / a.page_size : static_cast<unsigned>(slot) / static_cast<unsigned>(a.page_size);
            if (page < a.num_pages) row0 = (page * a.H + h0) * a.page_size + (slot - page * a.page_size);
            else if (lane == 0) atomicOr(a.status, kStatusBadCacheIndex);
        }
    }
    if (kind < 2) {
        // cos and sin of this lane's features: HALVES: of feature i mod turned / 2; else of pair i / 2
        const int half = a.turned / 2;
        const bool turns = lane * 8 < a.turned, first = lane * 8 < half;
        constexpr int NC = HALVES ? 8 : 4;
        float c[NC], s[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) c[j] = 1.f, s[j] = 0.f;
        if (known && turns) {
            const float* tab = a.rotation + pos * a.turned + (HALVES ? (first ? lane * 8 : lane * 8 - half) : lane * 4);
#pragma unroll
            for (int j = 0; j < NC; j += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4*>(tab + j)), w = __ldg(reinterpret_cast<const float4*>(tab + half + j));
                c[j] = u.x, c[j + 1] = u.y, c[j + 2] = u.z, c[j + 3] = u.w;
                s[j] = w.x, s[j + 1] = w.y, s[j + 2] = w.z, s[j + 3] = w.w;
            }
        }
        if (HALVES && first) {  // the first of a pair: a cos + b (-sin); the second: b cos + a sin
#pragma unroll
            for (int j = 0; j < NC; ++j) s[j] = -s[j];
        }
        const int base = threadIdx.x & 31 & ~(LANES - 1);
        const int partner = base + (turns ? (first ? lane + half / 8 : lane - half / 8) : lane);
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
            if (i >= heads) break;  // the same for the whole CTA
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 p = attn::unpack2<F16>(w[j]);
                float r0, r1;
                if constexpr (HALVES) {
                    const float2 o = attn::unpack2<F16>(__shfl_sync(kFullMask, w[j], partner));
                    r0 = __fadd_rn(__fmul_rn(p.x, c[2 * j]), __fmul_rn(o.x, s[2 * j]));
                    r1 = __fadd_rn(__fmul_rn(p.y, c[2 * j + 1]), __fmul_rn(o.y, s[2 * j + 1]));
                } else {
                    r0 = __fsub_rn(__fmul_rn(p.x, c[j]), __fmul_rn(p.y, s[j]));
                    r1 = __fadd_rn(__fmul_rn(p.y, c[j]), __fmul_rn(p.x, s[j]));
                }
                if (turns) w[j] = attn::pack2<F16>(r0, r1);  // what is not turned keeps its bits
            }
            x[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (kind == 0) {
        uint16_t* dst = a.q_out + t * a.q_out_stride + h0 * D + lane * 8;
#pragma unroll
        for (int i = 0; i < HEADS; ++i)
            if (known && i < heads) __stcs(reinterpret_cast<uint4*>(dst + i * D), x[i]);
        return;
    }
    uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? a.kc : a.vc) + (row0 * D + lane * 8) * (F8 ? 1 : 2);
    const long long step = static_cast<long long>(a.page_size) * D * (F8 ? 1 : 2);
    float* scales = (kind == 1 ? a.ks : a.vs) + row0;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        if (i >= heads) break;
        if constexpr (F8) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            float scale;
            const uint2 q = quantise8<LANES, F16>(w, scale);
            if (row0 >= 0) {
                *reinterpret_cast<uint2*>(dst + i * step) = q;
                if (lane == 0) scales[static_cast<long long>(i) * a.page_size] = scale;
            }
        } else if (row0 >= 0) {
            *reinterpret_cast<uint4*>(dst + i * step) = x[i];
        }
    }
}

}  // namespace cache
}  // namespace gdn
