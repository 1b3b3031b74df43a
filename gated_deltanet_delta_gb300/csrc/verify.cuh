// verify.cuh -- verification of drafted tokens (rejection sampling) from given random numbers.
//
// Sequence n has T drafted tokens x_t, the draft's distribution q_t that each was drawn from and the
// target's p_0 .. p_T.  Token t is accepted while u_t q_t(x_t) < p_t(x_t); at the first rejection r one
// token is drawn from max(p_r - q_r, 0) normalised, after T acceptances from p_T, so that what comes out
// is distributed as the target.  The draw inverts the cumulative distribution in whole units of 2^-36:
//     P_i = floor(min(max(p_i, 0), 1) 2^36), Q_i likewise;  w_i = max(P_i - Q_i, 0)  (P_i where all are 0);
//     mark = floor(sum w * floor(u 2^24) / 2^24);  token = the least i with w_0 + .. + w_i > mark.
// Integer sums do not depend on their order, so the token is a function of the inputs alone, whatever
// the division among threads; what the floor takes off is at most V 2^-36 of the mass.
//
// Bound: one row of p, and of q after a rejection, is read once.  HBM in the limit; one sequence is a chain of
// dependent loads, and a batch has such a chain at each wave's beginning and a last wave that is not full (255 sequences
// in clusters of four are 1.7 waves).  A cluster of CTAs takes a sequence: each sums its part of the row by chunks of 256
// entries and writes its sum into every CTA's shared memory, and the one CTA whose part holds the mark
// finds the chunk and reads its 256 entries again (from L2) while the others are already gone.  One launch, no workspace, no atomics.
// Measured: 3 drafts, 255 sequences, 100003 entries, 204 MB: 44 us, 4.6 TB/s; 4 drafts, one sequence: 6.9 us.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernel_args.h"

namespace gdn {
namespace verify {

constexpr int kThreads = 256;
constexpr int kChunk = 256;            // entries per chunk: eight per lane
typedef unsigned long long u64;

// P = floor(x 2^36) of a value in [0, 1] as P = hi 2^18 + lo, each plus 0x4B000000 (the bits of 2^23):
// adding 2^23 with truncation leaves a number's whole part in the significand.  Float additions run at
// full rate; a conversion to 64-bit integers took 50 cycles per warp and four fifths of the kernel's time.
struct Units {
    int hi, lo;
};
__device__ __forceinline__ Units units(float x) {
    const float h = __fmaf_rz(x, 262144.f, 8388608.f);
    const float rest = __fmaf_rn(x, 262144.f, 8388608.f - h);  // exact, in [0, 1)
    return {__float_as_int(h), __float_as_int(__fmaf_rz(rest, 262144.f, 8388608.f))};
}
// Adds max(P - Q, 0) to hi 2^18 + lo.  x > y implies P >= Q; NaN counts as 0.
__device__ __forceinline__ void add_weight(float x, float y, int& hi, int& lo) {
    x = __saturatef(x);
    y = __saturatef(y);
    const Units a = units(x), b = units(y);
    if (x > y) {
        hi += a.hi - b.hi;
        lo += a.lo - b.lo;
    }
}
__device__ __forceinline__ u64 joined(int hi, int lo) { return static_cast<u64>((static_cast<long long>(hi) << 18) + lo); }
__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(const __grid_constant__ VerifyArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ u64 sums[];        // this CTA's chunks
    __shared__ u64 total_s[2][8];        // every CTA's total, by rank, of the two passes
    __shared__ int count_s, drafts_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int n = blockIdx.x / C;
    // A CTA may write into another's shared memory only when that one has begun; waited for below, behind the row
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");

    if (warp == 0) {  // every CTA of the cluster counts for itself
        const long long given = a.num_drafts ? a.num_drafts[n] : a.T;
        const int T = static_cast<int>(min(max(given, 0LL), static_cast<long long>(a.T)));
        int count = T;
        for (int t0 = 0; t0 < T; t0 += 32) {
            const int t = t0 + lane;
            bool ok = true;
            if (t < T) {
                const long long x = a.drafts[static_cast<long long>(n) * a.T + t];
                if (x < 0 || x >= a.V) {
                    ok = false;
                    if (rank == 0) atomicOr(a.status, kStatusBadToken);
                } else {
                    const float p = a.target[(static_cast<long long>(n) * (a.T + 1) + t) * a.V + x];
                    const float q = a.draft[(static_cast<long long>(n) * a.T + t) * a.V + x];
                    ok = __fmul_rn(a.u_accept[static_cast<long long>(n) * a.T + t], q) < p;
                }
            }
            const unsigned no = __ballot_sync(kFullMask, !ok);
            if (no) {
                count = t0 + __ffs(no) - 1;
                break;
            }
        }
        if (lane == 0) {
            count_s = count;
            drafts_s = T;
        }
    }
    __syncthreads();
    const int count = count_s;
    const float* p = a.target + (static_cast<long long>(n) * (a.T + 1) + count) * a.V;
    const float* q = count < drafts_s ? a.draft + (static_cast<long long>(n) * a.T + count) * a.V : nullptr;

    // this CTA's chunks of the row
    const int chunks = (a.V + kChunk - 1) / kChunk;
    const int c0 = static_cast<int>(static_cast<long long>(chunks) * rank / C);
    const int c1 = static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / C);
    u64 mine = 0, all = 0, before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        mine = 0;
        // one chunk ahead: a warp's next sixteen loads are in flight while it adds up this one's
        float x[8], y[8], xn[8], yn[8];
        auto load = [&](int c, float (&u)[8], float (&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = c * kChunk + j * 32 + lane;
                const bool in = c < c1 && i < a.V;
                u[j] = in ? p[i] : 0.f;
                v[j] = q && in ? q[i] : 0.f;
            }
        };
        load(c0 + warp, x, y);
        for (int c = c0 + warp; c < c1; c += kThreads / 32) {
            load(c + kThreads / 32, xn, yn);
            int hi = 0, lo = 0;  // 256 entries of at most 2^18: no overflow
#pragma unroll
            for (int j = 0; j < 8; ++j) add_weight(x[j], y[j], hi, lo);
            const u64 s = joined(__reduce_add_sync(kFullMask, hi), __reduce_add_sync(kFullMask, lo));
            if (lane == 0) sums[c - c0] = s;
            mine += s;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = xn[j];
                y[j] = yn[j];
            }
        }
        __shared__ u64 warp_s[kThreads / 32];
        if (lane == 0) warp_s[warp] = mine;
        __syncthreads();
        mine = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) mine += warp_s[i];
        if (pass == 0) asm volatile("barrier.cluster.wait;" ::: "memory");
        if (tid < C) *cluster.map_shared_rank(&total_s[pass][rank], tid) = mine;
        cluster.sync();
        all = before = 0;
        for (int r = 0; r < C; ++r) {
            const u64 s = total_s[pass][r];
            all += s;
            if (r < rank) before += s;
        }
        if (all > 0 || !q) break;  // the same for the whole cluster
        q = nullptr;               // the draft covers all of p: draw from p itself
        __syncthreads();
    }

    const float u = a.u_sample[n];
    const u64 u24 = static_cast<u64>(fminf(fmaxf(u, 0.f), 16777215.f / 16777216.f) * 16777216.f);
    // all * u24 may pass 64 bits where rows are far from normalised: the product's bits 24 ..
    const u64 mark = __umul64hi(all, u24) << 40 | (all * u24) >> 24;
    int64_t* out = a.tokens + static_cast<long long>(n) * (a.T + 1);
    if (warp == 0 && all > 0 && mark >= before && mark - before < mine) {
        u64 left = mark - before;
        int c = 0;
        for (int b = 0; b < c1 - c0; b += 32) {  // the chunk that holds the mark
            const u64 s = b + lane < c1 - c0 ? sums[b + lane] : 0;
            const u64 inc = warp_scan(s, lane);
            const unsigned hit = __ballot_sync(kFullMask, inc > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                c = b + l;
                left -= __shfl_sync(kFullMask, inc - s, l);
                break;
            }
            left -= __shfl_sync(kFullMask, inc, 31);
        }
        const int i0 = (c0 + c) * kChunk;
        u64 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * 32 + lane;
            int hi = 0, lo = 0;
            if (i < a.V) add_weight(p[i], q ? q[i] : 0.f, hi, lo);
            w[j] = joined(hi, lo);
        }
        int token = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const u64 inc = warp_scan(w[j], lane);
            const unsigned hit = __ballot_sync(kFullMask, inc > left);
            if (token < 0) {
                if (hit) token = i0 + j * 32 + __ffs(hit) - 1;
                else left -= __shfl_sync(kFullMask, inc, 31);
            }
        }
        if (lane == 0) out[count] = token;
    }
    if (rank == 0) {
        if (tid == 0) {
            a.accepted[n] = count;
            if (all == 0) {  // the row holds nothing: token 0, and the status says so
                out[count] = 0;
                atomicOr(a.status, kStatusBadProbs);
            }
        }
        for (int t = tid; t <= a.T; t += kThreads)
            if (t != count) out[t] = t < count ? a.drafts[static_cast<long long>(n) * a.T + t] : -1;
    }
}

}  // namespace verify
}  // namespace gdn
