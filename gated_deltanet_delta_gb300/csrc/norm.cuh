// norm.cuh -- root-mean-square norm with the residual's addition:
//     r = x + residual (rounded to the rows' type, and stored: the residual stream);   y = r / sqrt(mean(r^2) + eps) * w,
// in the rows' type, or in e4m3 with scale = max |y| / 448 for each group of features (1 where all are zero, at least
// 2^-126): for the operand of a product in 8 bits the whole range is used; a power of two would leave up to half of it.
//
// Each value is read once and written once: the bound is HBM.  blockDim.x threads hold a row in registers, R
// pieces of eight features each, blockDim.y short rows per CTA.  The sum of squares is taken over the rounded r, in fp32.
// A row waits for its loads and then for its sums, so what counts is how many rows an SM has at once: 32 registers a thread, one or two
// pieces.  Measured, 16383 rows of 5120, bf16 to e4m3 by groups of 128: 100 us, 88 % of a copy's rate (122 us with four pieces a
// thread, 160 us with rows through a ring of bulk copies, 130 us with CTAs that stay and load the next row ahead).
#pragma once

#include <cuda_fp8.h>

#include "attn_mma.cuh"
#include "common.cuh"
#include "kernel_args.h"
#include "tile_util.cuh"

namespace gdn {
namespace norm {

constexpr int kMaxThreads = 512;

// Sum (or largest) over the row's threads; every thread gets it.  buf: 32 floats per row.
template <bool MAX>
__device__ __forceinline__ float row_join(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(kFullMask, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (blockDim.x == 32) return v;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    v = lane < warps ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(kFullMask, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

template <bool F16>
__device__ __forceinline__ attn::f32x2 widen(uint32_t w) {
    if constexpr (!F16) return attn::widen2(w);
    const float2 f = attn::unpack2<F16>(w);
    return attn::pair(f.x, f.y);
}
// amax / 448: the product with 1 / 448 and what that leaves.
__device__ __forceinline__ float scale_of(float amax) {
    const float q = amax * (1.f / 448.f);
    return amax > 0.f ? fmaxf(fmaf(fmaf(-448.f, q, amax), 1.f / 448.f, q), 1.17549435e-38f) : 1.f;
}
// Eight values over the scale to e4m3: the quotient is the product with up, about 1 / scale, and what that leaves times up again, which makes it fp32's
// (by the product alone a quotient within 2^-22 of the middle between two went to either; divisions took 22 us more).
__device__ __forceinline__ uint2 to_e4m3(const float (&f)[8], float scale, float up) {
    uint32_t q[4];
    const attn::f32x2 ss = attn::pair(-scale, -scale), uu = attn::pair(up, up);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float g[2];
        const attn::f32x2 y = attn::pair(f[2 * j], f[2 * j + 1]), p = attn::mul2(y, uu);
        attn::unpair(attn::fma2(attn::fma2(p, ss, y), uu, p), g);
        q[j] = __nv_cvt_float2_to_fp8x2(make_float2(g[0], g[1]), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// What a thread does with its pieces of row t: x, r in; the residual, y and the scales out.  The joins take part in the
// CTA's barriers, so every thread comes here (`here`: whether it has a row).
template <bool F16, bool F8, int R>
__device__ __forceinline__ void row(const NormArgs& a, long long t, bool here, uint4 (&x)[R], const uint4 (&r)[R], float* sums, float* tops) {
    const int pieces = a.C / 8;
    auto piece = [&](int i) { return static_cast<int>(threadIdx.x + i * blockDim.x); };
    attn::f32x2 sums2 = attn::pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        const uint32_t v[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (a.residual) {
                float f[2];
                attn::unpair(attn::add2(widen<F16>(v[j]), widen<F16>(u[j])), f);
                u[j] = attn::pack2<F16>(f[0], f[1]);
            }
            const attn::f32x2 f = widen<F16>(u[j]);
            sums2 = attn::fma2(f, f, sums2);
        }
        x[i] = make_uint4(u[0], u[1], u[2], u[3]);
        if (a.residual && here && piece(i) < pieces) *reinterpret_cast<uint4*>(a.residual + t * a.C + piece(i) * 8) = x[i];
    }
    float sum[2];
    attn::unpair(sums2, sum);
    const float inv = rsqrtf(row_join<false>(sum[0] + sum[1], sums) / static_cast<float>(a.C) + a.eps);
    auto normed = [&](int i, float (&f)[8]) {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
        if (piece(i) < pieces) {
            p = __ldg(reinterpret_cast<const float4*>(a.w + piece(i) * 8));
            q = __ldg(reinterpret_cast<const float4*>(a.w + piece(i) * 8 + 4));
        }
        const attn::f32x2 w[4] = {attn::pair(p.x, p.y), attn::pair(p.z, p.w), attn::pair(q.x, q.y), attn::pair(q.z, q.w)};
        const attn::f32x2 by = attn::pair(inv, inv);
#pragma unroll
        for (int j = 0; j < 4; ++j) attn::unpair(attn::mul2(attn::mul2(widen<F16>(u[j]), by), w[j]), f + 2 * j);
    };
    float amax = 0.f;  // of the row (one scale per row)
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int p = piece(i);
        const bool on = here && p < pieces;
        float f[8];
        normed(i, f);
        if constexpr (!F8) {
            if (on)
                __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + t * a.C + p * 8),
                       make_uint4(attn::pack2<F16>(f[0], f[1]), attn::pack2<F16>(f[2], f[3]), attn::pack2<F16>(f[4], f[5]), attn::pack2<F16>(f[6], f[7])));
        } else {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
            if (a.lanes == 0) {
                amax = fmaxf(amax, m);
            } else {
                for (int o = a.lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
                const float scale = scale_of(m);
                if (on) {
                    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + t * a.C + p * 8), to_e4m3(f, scale, attn::fast_rcp(scale)));
                    if (p % a.lanes == 0) a.scale[t * (pieces / a.lanes) + p / a.lanes] = scale;
                }
            }
        }
    }
    if constexpr (F8) {
        if (a.lanes == 0) {
            amax = row_join<true>(amax, tops);
            const float scale = scale_of(amax), up = attn::fast_rcp(scale);
            if (here && threadIdx.x == 0) a.scale[t] = scale;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (!here || piece(i) >= pieces) continue;
                float f[8];
                normed(i, f);
                __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + t * a.C + piece(i) * 8), to_e4m3(f, scale, up));
            }
        }
    }
}

template <bool F16, bool F8, int R>
__global__ void __launch_bounds__(R == 1 ? 256 : kMaxThreads, R == 1 ? 6 : R == 2 ? 4 : 1) add_rms_norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float buf[2][8][32];
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool here = t < a.T;
    uint4 x[R], r[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int p = threadIdx.x + i * blockDim.x;
        const bool on = here && p < a.C / 8;
        x[i] = on ? *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + p * 8) : make_uint4(0, 0, 0, 0);
        r[i] = on && a.residual ? *reinterpret_cast<const uint4*>(a.residual + t * a.C + p * 8) : make_uint4(0, 0, 0, 0);
    }
    row<F16, F8, R>(a, t, here, x, r, buf[0][threadIdx.y], buf[1][threadIdx.y]);
}

}  // namespace norm
}  // namespace gdn
