// conv.cuh -- the short causal convolution of packed sequences, channel by channel:
//     y[t, c] = act(bias_c + sum_j w[c, j] x[t - (TAPS - 1) + j, c]),   act(y) = y / (1 + e^-y) or y,
// where the tokens ahead of a sequence's first are its history, TAPS - 1 values per channel that the pool keeps from call
// to call (oldest first, the layout that the decode window's history has).
//
// Each value is read once and written once: the bound is HBM.  A thread has eight channels (16-byte accesses) of consecutive tokens,
// with the weights in registers; the TAPS - 1 tokens ahead of its tile come from L2, where the tile before read them.  Short calls go
// in tiles of 32 tokens, the next eight of them loaded ahead (short_conv_kernel); long ones in tiles of 128 whose rows arrive through
// a ring of bulk copies, so that many bytes are on their way with few registers (short_conv_ring_kernel; 23508 tokens of 8192
// channels, bf16: 140 us, 82 % of a copy's rate; 154 us with the loads of the other, 145 us with four stages and three CTAs per SM, 151
// us with two stages and five).  What is left above the 115 us of the bytes is the latency of sixteen warps' arithmetic: 47 % of the
// issue slots, a value's own dependences the largest stall.
//
// The new history is written by a kernel of its own behind the first: in the same one, the CTA that reaches a sequence's end would
// overwrite what the CTA at its start has yet to read.  A step of one token per sequence has no such order to keep, and is one launch.
#pragma once

#include "attn_mma.cuh"
#include "common.cuh"
#include "kernel_args.h"
#include "tcgen05.cuh"
#include "tile_util.cuh"

namespace gdn {
namespace conv {

constexpr int kThreads = 128;
constexpr int kTokens = 32;
constexpr int kStep = 8;  // tokens in registers, and as many on their way
// the kernel for long calls
constexpr int kTile = 128;
constexpr int kStages = 3;
constexpr int kRing = kStages * kStep * kThreads * 16;
constexpr uint32_t kWaitPolls = 1u << 24;  // the built-in limit of a wait for a copy (seconds)
static_assert(kTile == kThreads, "a thread per token");

// A token's sequence: which, where it begins and ends; n = -1 for a token of no (well-formed) sequence.
struct Place {
    long long begin, end;
    int n;
};
__device__ __forceinline__ Place place_of(const int64_t* cu, int num_seqs, long long T, long long t) {
    int lo = 0, hi = num_seqs;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    Place p{cu[lo], cu[lo + 1], lo};
    if (p.begin < 0 || p.begin > t || t >= p.end || p.end > T) p.n = -1;
    return p;
}

using attn::f32x2;

// Eight channels as pairs.
template <int TAPS>
struct Weights {
    f32x2 w[TAPS][4], b[4];
    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
        float f[8 * TAPS];
        const float4* src = reinterpret_cast<const float4*>(a.w + static_cast<long long>(c) * TAPS);
#pragma unroll
        for (int i = 0; i < 2 * TAPS; ++i) reinterpret_cast<float4*>(f)[i] = __ldg(src + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < TAPS; ++j) w[j][i] = attn::pair(f[2 * i * TAPS + j], f[(2 * i + 1) * TAPS + j]);
            b[i] = a.bias ? attn::pair(__ldg(a.bias + c + 2 * i), __ldg(a.bias + c + 2 * i + 1)) : attn::pair(0.f, 0.f);
        }
    }
};

// TAPS - 1 values of each of eight channels, oldest first.
template <int TAPS>
struct Past {
    f32x2 v[TAPS - 1][4];
    __device__ __forceinline__ void load(const float* hist) {
        float f[8 * (TAPS - 1)];
#pragma unroll
        for (int i = 0; i < 2 * (TAPS - 1); ++i) reinterpret_cast<float4*>(f)[i] = reinterpret_cast<const float4*>(hist)[i];
#pragma unroll
        for (int j = 0; j < TAPS - 1; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = attn::pair(f[2 * i * (TAPS - 1) + j], f[(2 * i + 1) * (TAPS - 1) + j]);
    }
    __device__ __forceinline__ void store(float* hist) const {
        float f[8 * (TAPS - 1)], u[2];
#pragma unroll
        for (int j = 0; j < TAPS - 1; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                attn::unpair(v[j][i], u);
                f[2 * i * (TAPS - 1) + j] = u[0];
                f[(2 * i + 1) * (TAPS - 1) + j] = u[1];
            }
#pragma unroll
        for (int i = 0; i < 2 * (TAPS - 1); ++i) reinterpret_cast<float4*>(hist)[i] = reinterpret_cast<const float4*>(f)[i];
    }
    __device__ __forceinline__ void push(const f32x2 (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j + 1 < TAPS - 1; ++j) v[j][i] = v[j + 1][i];
            v[TAPS - 2][i] = x[i];
        }
    }
};

template <bool F16>
__device__ __forceinline__ void widen8(const uint4& p, f32x2 (&f)[4]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 u = attn::unpack2<F16>(w[j]);
        f[j] = attn::pair(u.x, u.y);
    }
}

// One token's eight outputs.
template <int TAPS, bool F16>
__device__ __forceinline__ uint4 token(const Weights<TAPS>& w, const Past<TAPS>& p, const f32x2 (&x)[4], bool silu) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f32x2 y = w.b[i];
#pragma unroll
        for (int j = 0; j < TAPS - 1; ++j) y = attn::fma2(w.w[j][i], p.v[j][i], y);
        y = attn::fma2(w.w[TAPS - 1][i], x[i], y);
        if (silu) y = attn::silu2_joint(y);
        float f[2];
        attn::unpair(y, f);
        r[i] = attn::pack2<F16>(f[0], f[1]);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Where channel c of token 0 goes, and the distance between tokens.
__device__ __forceinline__ uint16_t* out_of(const ConvArgs& a, int c, int& width) {
    const int i = c < a.width[0] ? 0 : c < a.width[0] + a.width[1] ? 1 : 2;
    width = a.width[i];
    return a.out[i] + (c - (i > 0 ? a.width[0] : 0) - (i > 1 ? a.width[1] : 0));
}

// What is ahead of a tile: its first token's sequence's tokens (`ahead` of them), and before those the history.
template <int TAPS, bool F16>
__device__ __forceinline__ void ahead_of_tile(const ConvArgs& a, Past<TAPS>& p, const uint16_t* src, int c, long long slot, int ahead) {
    if (slot >= 0 && ahead < TAPS - 1) {
        p.load(a.hist + (slot * a.C + c) * (TAPS - 1));
    } else {
#pragma unroll
        for (int j = 0; j < TAPS - 1; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.v[j][i] = attn::pair(0.f, 0.f);
    }
    for (int j = slot >= 0 ? ahead : 0; j > 0; --j) {
        f32x2 f[4];
        widen8<F16>(*reinterpret_cast<const uint4*>(src - j * a.x_stride), f);
        p.push(f);
    }
}

// One token per sequence: outputs, and the history in place.
template <int TAPS, bool F16>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const __grid_constant__ ConvArgs a) {
    const int n = blockIdx.x, c = (blockIdx.y * kThreads + threadIdx.x) * 8;
    const long long slot = a.slots[n];
    if (slot < 0 || slot >= a.pool_size) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadCacheIndex);
        return;
    }
    if (c >= a.C) return;
    f32x2 x[4];
    widen8<F16>(__ldcs(reinterpret_cast<const uint4*>(a.x + n * a.x_stride + c)), x);
    float* hist = a.hist + (slot * a.C + c) * (TAPS - 1);
    Past<TAPS> p;
    p.load(hist);
    Weights<TAPS> w;
    w.load(a, c);
    int width;
    uint16_t* out = out_of(a, c, width);
    *reinterpret_cast<uint4*>(out + static_cast<long long>(n) * width) = token<TAPS, F16>(w, p, x, a.silu);
    p.push(x);
    p.store(hist);
}

template <int TAPS, bool F16>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const __grid_constant__ ConvArgs a) {
    __shared__ long long slot_s[kTokens];  // of each token; -1: of no (well-formed) sequence
    __shared__ int ahead_s[kTokens];       // tokens of its sequence ahead of it, at most TAPS - 1
    const int c = (blockIdx.y * kThreads + threadIdx.x) * 8;
    const long long t0 = static_cast<long long>(blockIdx.x) * kTokens;
    const int count = static_cast<int>(a.T - t0 < kTokens ? a.T - t0 : kTokens);
    const bool on = c < a.C;
    const uint16_t* src = a.x + t0 * a.x_stride + c;
    auto fetch = [&](uint4 (&x)[kStep], int i0) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            x[i] = on && i0 + i < count ? *reinterpret_cast<const uint4*>(src + (i0 + i) * a.x_stride) : make_uint4(0, 0, 0, 0);
    };
    uint4 x[kStep], next[kStep];
    fetch(x, 0);
    int odd = 0;  // whether the token begins a sequence, or belongs to none
    if (threadIdx.x < kTokens) {
        const int i = threadIdx.x;
        long long slot = -1;
        int ahead = 0;
        if (i < count) {
            const Place p = place_of(a.cu, a.num_seqs, a.T, t0 + i);
            if (p.n >= 0) {
                slot = a.slots[p.n];
                if (slot < 0 || slot >= a.pool_size) slot = -1;  // reported by the history's kernel
                ahead = static_cast<int>(t0 + i - p.begin < TAPS - 1 ? t0 + i - p.begin : TAPS - 1);
            }
        }
        slot_s[i] = slot;
        ahead_s[i] = ahead;
        odd = slot < 0 || (i > 0 && ahead == 0);
    }
    const bool plain = !__syncthreads_or(odd);  // one sequence throughout
    if (!on) return;
    Weights<TAPS> w;
    w.load(a, c);
    int width;
    uint16_t* out = out_of(a, c, width) + t0 * width;
    Past<TAPS> p;
    ahead_of_tile<TAPS, F16>(a, p, src, c, slot_s[0], ahead_s[0]);
    if (plain) {
#pragma unroll 1
        for (int i0 = 0; i0 < kTokens; i0 += kStep) {
            fetch(next, i0 + kStep);
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                f32x2 f[4];
                widen8<F16>(x[i], f);
                __stcs(reinterpret_cast<uint4*>(out + static_cast<long long>(i0 + i) * width), token<TAPS, F16>(w, p, f, a.silu));
                p.push(f);
                x[i] = next[i];
            }
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const long long slot = slot_s[i];
        if (i > 0 && ahead_s[i] == 0 && slot >= 0) p.load(a.hist + (slot * a.C + c) * (TAPS - 1));
        f32x2 f[4];
        widen8<F16>(*reinterpret_cast<const uint4*>(src + i * a.x_stride), f);
        if (slot >= 0) __stcs(reinterpret_cast<uint4*>(out + static_cast<long long>(i) * width), token<TAPS, F16>(w, p, f, a.silu));
        p.push(f);
    }
}

// The same for long calls: 128 tokens per CTA, whose rows come by bulk copies into a ring of kStages steps of eight tokens in shared memory.
// With the rows in registers there is room for 12 warps with eight loads each on an SM, and 72 % of HBM's rate.  A copy that
// does not arrive within the limit of a wait is done without: the thread reads its rows directly, and the CTA ends behind one more bounded
// wait for each copy that is still to come.
template <int TAPS, bool F16>
__global__ void __launch_bounds__(kThreads) short_conv_ring_kernel(const __grid_constant__ ConvArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];  // [kStages][kStep][kThreads * 8] elements
    __shared__ long long slot_s[kTile];
    __shared__ int ahead_s[kTile];
    __shared__ uint32_t odd_s[kTile / 32];  // tokens that begin a sequence, or belong to none
    __shared__ uint64_t full[kStages];
    constexpr uint32_t ROW = kThreads * 16, STAGE = kStep * ROW;
    const int c0 = blockIdx.y * kThreads * 8, c = c0 + threadIdx.x * 8;
    const long long t0 = static_cast<long long>(blockIdx.x) * kTile;
    const int count = static_cast<int>(a.T - t0 < kTile ? a.T - t0 : kTile), steps = (count + kStep - 1) / kStep;
    const bool on = c < a.C;
    const uint16_t* src = a.x + t0 * a.x_stride + c;
    const uint32_t bytes = static_cast<uint32_t>(min(kThreads * 8, a.C - c0)) * 2;
    auto issue = [&](int k) {  // by thread 0
        const int tokens = min(kStep, count - k * kStep), s = k % kStages;
        tc::mbar_expect_tx(&full[s], tokens * bytes);
        for (int i = 0; i < tokens; ++i)
            tc::bulk_load(tc::smem_u32(ring) + s * STAGE + i * ROW, a.x + (t0 + k * kStep + i) * a.x_stride + c0, bytes, &full[s]);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[s], 1);
        for (int k = 0; k < kStages && k < steps; ++k) issue(k);
    }
    {
        const int i = threadIdx.x;
        long long slot = -1;
        int ahead = 0;
        if (i < count) {
            const Place p = place_of(a.cu, a.num_seqs, a.T, t0 + i);
            if (p.n >= 0) {
                slot = a.slots[p.n];
                if (slot < 0 || slot >= a.pool_size) slot = -1;  // reported by the history's kernel
                ahead = static_cast<int>(t0 + i - p.begin < TAPS - 1 ? t0 + i - p.begin : TAPS - 1);
            }
        }
        slot_s[i] = slot;
        ahead_s[i] = ahead;
        const uint32_t odd = __ballot_sync(kFullMask, slot < 0 || (i > 0 && ahead == 0));
        if (i % 32 == 0) odd_s[i / 32] = odd;
    }
    __syncthreads();
    Weights<TAPS> w;
    Past<TAPS> p;
    int width = 0;
    uint16_t* out = nullptr;
    if (on) {
        w.load(a, c);
        out = out_of(a, c, width) + t0 * width;
        ahead_of_tile<TAPS, F16>(a, p, src, c, slot_s[0], ahead_s[0]);
    }
    const bool tight = a.polls < kWaitPolls;  // with the limit a variable in every wait: 141 us instead of 139
    bool ok = true;
    int unseen = steps;  // the first step whose copies this thread has not seen arrive
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        const int s = k % kStages, i0 = k * kStep;
        if (ok && !(tight ? tc::mbar_wait(&full[s], k / kStages & 1, a.polls) : tc::mbar_wait(&full[s], k / kStages & 1, kWaitPolls))) ok = false, unseen = k;
        const uint8_t* held = ring + s * STAGE + threadIdx.x * 16;
        auto row = [&](int i) {
            return ok ? *reinterpret_cast<const uint4*>(held + i * ROW) : *reinterpret_cast<const uint4*>(src + (i0 + i) * a.x_stride);
        };
        if (on) {
            if ((odd_s[i0 / 32] >> (i0 % 32) & 0xff) == 0) {
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    f32x2 f[4];
                    widen8<F16>(row(i), f);
                    __stcs(reinterpret_cast<uint4*>(out + static_cast<long long>(i0 + i) * width), token<TAPS, F16>(w, p, f, a.silu));
                    p.push(f);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kStep && i0 + i < count; ++i) {
                    const long long slot = slot_s[i0 + i];
                    if (i0 + i > 0 && ahead_s[i0 + i] == 0 && slot >= 0) p.load(a.hist + (slot * a.C + c) * (TAPS - 1));
                    f32x2 f[4];
                    widen8<F16>(row(i), f);
                    if (slot >= 0) __stcs(reinterpret_cast<uint4*>(out + static_cast<long long>(i0 + i) * width), token<TAPS, F16>(w, p, f, a.silu));
                    p.push(f);
                }
            }
        }
        __syncthreads();  // the step's place has been read
        if (threadIdx.x == 0 && ok && k + kStages < steps) issue(k + kStages);
    }
    if (threadIdx.x == 0)  // thread 0 issued no more once it had given up
        for (int k = unseen; k < min(unseen + kStages, steps); ++k) tc::mbar_wait(&full[k % kStages], k / kStages & 1, kWaitPolls);
}

// The history behind each sequence's last token, and the report of malformed bounds and slots.
template <int TAPS, bool F16>
__global__ void __launch_bounds__(kThreads) short_conv_history_kernel(const __grid_constant__ ConvArgs a) {
    const int n = blockIdx.x, c = (blockIdx.y * kThreads + threadIdx.x) * 8;
    const long long begin = a.cu[n], end = a.cu[n + 1], slot = a.slots[n];
    const bool bad = begin < 0 || end < begin || end > a.T, off = slot < 0 || slot >= a.pool_size;
    if (bad || off) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, (bad ? kStatusBadSeqlens : 0) | (off ? kStatusBadCacheIndex : 0));
        return;
    }
    if (c >= a.C || end == begin) return;
    float* hist = a.hist + (slot * a.C + c) * (TAPS - 1);
    Past<TAPS> p;
    if (end - begin < TAPS - 1) p.load(hist);
    const int fresh = static_cast<int>(end - begin < TAPS - 1 ? end - begin : TAPS - 1);
    for (int j = fresh; j > 0; --j) {
        f32x2 f[4];
        widen8<F16>(*reinterpret_cast<const uint4*>(a.x + (end - j) * a.x_stride + c), f);
        p.push(f);
    }
    p.store(hist);
}

}  // namespace conv
}  // namespace gdn
