// ssm.cuh -- the selective state space recurrence as it stands, token by token, for single tokens and short sequences:
//     dt_t = softplus(raw_t + bias);  S_t = e^(A dt_t) S_(t-1) + dt_t x_t (x) B_t,  A = -e^A_log;
//     y_t = S_t C_t + D x_t, times silu(z_t) where there is a gate.
// Head h has P features and reads B and C of group h / (H / G); its state is [P, N], in fp32.
//
// A stream of the state, 8 bytes per element and call against 4 operations per token: HBM is the bound up to some ten
// tokens.  A state row of N floats is split over TPR lanes, a thread has two rows and asks for all of its 16-byte pieces
// before any arithmetic (as gdn_decode_kernel does); the tokens' inputs are staged in shared memory, kSteps at a time.
// CTAs of 32 rows: while some load, others compute and store (of 64 rows: 48.9 and 36.9 us).  Measured, one token of 64 sequences, 64
// heads of 64, N = 128 (270 MB): 45.1 us, 89 % of a copy's rate; 32 sequences of up to 8 tokens, no gate: 32.8 us, 62 %, where no unit is
// the limit: a scheduler issues in 49 % of the cycles, and its warps wait for the state, for shared memory and shuffles (a sum over lanes
// for each output), and for the instruction before, in about equal parts.
#pragma once

#include "common.cuh"
#include "kernel_args.h"
#include "tile_util.cuh"

namespace gdn {
namespace ssm {

constexpr int kSteps = 8;    // tokens staged at a time
constexpr int kRows = 32;    // state rows per CTA

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
// z / (1 + e^-z) as z e^z / (1 + e^z), e^z held at e^40: both ends of z's range stay in it, and go to 0 and to z.
__device__ __forceinline__ float silu(float z) {
    const float t = __expf(fminf(z, 40.f));
    return z * __fdividef(t, 1.f + t);
}

// The bounds and the slot of sequence n; false (and the status) if they are malformed.
__device__ __forceinline__ bool sequence(const SsmArgs& a, int n, long long& begin, long long& end, long long& slot, bool report) {
    begin = a.cu ? a.cu[n] : n;
    end = a.cu ? a.cu[n + 1] : n + 1;
    slot = a.slots[n];
    const bool bad = begin < 0 || end < begin || end > a.T, off = slot < 0 || slot >= a.pool_size;
    if ((bad || off) && report) atomicOr(a.status, (bad ? kStatusBadSeqlens : 0) | (off ? kStatusBadCacheIndex : 0));
    return !bad && !off;
}

// ONE: one token per sequence.  Without the loop over tokens it takes fewer registers, and three CTAs fit an SM.
template <int S, int TPR, bool ONE>
__global__ void __launch_bounds__(kRows / 2 * TPR, 768 / (kRows / 2 * TPR)) ssm_steps_kernel(const __grid_constant__ SsmArgs a) {
    constexpr int NT = kRows / 2 * TPR, NV = S / (4 * TPR), RPP = NT / TPR, STEPS = ONE ? 1 : kSteps;
    __shared__ float4 Bs[STEPS][S / 4], Cs[STEPS][S / 4];
    __shared__ float xs[STEPS][kRows], keep_s[STEPS], dt_s[STEPS];
    const int tile = blockIdx.x % a.tiles, h = blockIdx.x / a.tiles % a.H, n = blockIdx.x / a.tiles / a.H;
    const int g = h / (a.H / a.G), p0 = tile * kRows;
    const int lr = threadIdx.x % TPR, rw = threadIdx.x / TPR;
    long long begin, end, slot;
    if (!sequence(a, n, begin, end, slot, threadIdx.x == 0 && tile == 0 && h == 0) || begin == end) return;
    float4* st = reinterpret_cast<float4*>(a.state) + ((slot * a.H + h) * a.P + p0) * (S / 4);
    float4 s[2][NV];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int m = 0; m < NV; ++m) s[r][m] = ld_stream(st + (r * RPP + rw) * (S / 4) + lr + TPR * m);
    const float A = -expf(a.A_log[h]), bias = a.dt_bias[h], D = a.D ? a.D[h] : 0.f;
    for (long long t0 = begin; t0 < end; t0 += STEPS) {
        const int count = ONE ? 1 : static_cast<int>(end - t0 < STEPS ? end - t0 : STEPS);
        if (!ONE && t0 > begin) __syncthreads();  // the block before is no longer read
        for (int i = threadIdx.x; i < count * (S / 4); i += NT) {
            const int k = i / (S / 4), j = i % (S / 4);
            Bs[k][j] = bf16x4_to_f32x4(*reinterpret_cast<const uint2*>(a.B + (t0 + k) * a.b_stride + g * S + 4 * j));
            Cs[k][j] = bf16x4_to_f32x4(*reinterpret_cast<const uint2*>(a.C + (t0 + k) * a.c_stride + g * S + 4 * j));
        }
        for (int i = threadIdx.x; i < count * kRows; i += NT)
            xs[i / kRows][i % kRows] = bf16_to_f32(a.x[(t0 + i / kRows) * a.x_stride + h * a.P + p0 + i % kRows]);
        if (threadIdx.x < count) {
            const float dt = softplus(bf16_to_f32(a.dt[(t0 + threadIdx.x) * a.dt_stride + h]) + bias);
            dt_s[threadIdx.x] = dt;
            keep_s[threadIdx.x] = expf(A * dt);
        }
        __syncthreads();
        for (int k = 0; k < count; ++k) {
            const float keep = keep_s[k], dt = dt_s[k];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r * RPP + rw;
                const float x = xs[k][row], add = dt * x;
                float y = 0.f;
                attn::f32x2 yy = attn::pair(0.f, 0.f);
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    const float4 b = Bs[k][lr + TPR * m], c = Cs[k][lr + TPR * m];
                    float4& v = s[r][m];
                    if constexpr (ONE) {
                        v.x = fmaf(keep, v.x, add * b.x);
                        v.y = fmaf(keep, v.y, add * b.y);
                        v.z = fmaf(keep, v.z, add * b.z);
                        v.w = fmaf(keep, v.w, add * b.w);
                        y += dot4(v, c);
                    } else {  // in pairs: the arithmetic of several tokens counts
                        const attn::f32x2 kk = attn::pair(keep, keep), aa = attn::pair(add, add);
                        const attn::f32x2 p = attn::fma2(kk, attn::pair(v.x, v.y), attn::mul2(aa, attn::pair(b.x, b.y)));
                        const attn::f32x2 q = attn::fma2(kk, attn::pair(v.z, v.w), attn::mul2(aa, attn::pair(b.z, b.w)));
                        yy = attn::fma2(p, attn::pair(c.x, c.y), attn::fma2(q, attn::pair(c.z, c.w), yy));
                        float f[4];
                        attn::unpair(p, f);
                        attn::unpair(q, f + 2);
                        v = make_float4(f[0], f[1], f[2], f[3]);
                    }
                }
                if constexpr (!ONE) {
                    float f[2];
                    attn::unpair(yy, f);
                    y = f[0] + f[1];
                }
                y = fmaf(D, x, group_sum<TPR>(y));
                if (lr == 0) {
                    const long long at = h * a.P + p0 + row;
                    if (a.z) y *= silu(bf16_to_f32(a.z[(t0 + k) * a.z_stride + at]));
                    a.out[(t0 + k) * a.H * a.P + at] = f32_to_bf16_rne(y);
                }
            }
        }
        if (ONE) break;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int m = 0; m < NV; ++m) st_stream(st + (r * RPP + rw) * (S / 4) + lr + TPR * m, s[r][m]);
}

}  // namespace ssm
}  // namespace gdn
