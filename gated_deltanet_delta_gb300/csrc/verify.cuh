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
// Bound: one row of p, and of q after a rejection, is read once: HBM for a batch, latency for one
// sequence.  A cluster of CTAs takes a sequence: each sums its part of the row by chunks of 256
// entries, the parts' sums cross the cluster's shared memory, and the one CTA whose part holds the mark
// finds the chunk and reads its 256 entries again (from L2).  One launch, no workspace, no atomics.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernel_args.h"

namespace gdn {
namespace verify {

constexpr int kThreads = 512;
constexpr int kChunk = 256;            // entries per chunk: eight per lane
constexpr int kMaxChunks = 4096;       // per CTA
typedef unsigned long long u64;

__device__ __forceinline__ u64 units(float p) {
    return __float2ull_rz(fminf(fmaxf(p, 0.f), 1.f) * 68719476736.f);  // NaN counts as 0
}
__device__ __forceinline__ u64 weight(float p, float q) {
    const u64 a = units(p), b = units(q);
    return a > b ? a - b : 0;
}
__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
    return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const __grid_constant__ VerifyArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ u64 sums[];        // this CTA's chunks
    __shared__ u64 total_s[2];
    __shared__ int count_s, drafts_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int n = blockIdx.x / C;

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
        for (int c = c0 + warp; c < c1; c += kThreads / 32) {
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = c * kChunk + j * 32 + lane;
                x[j] = i < a.V ? p[i] : 0.f;
                y[j] = q && i < a.V ? q[i] : 0.f;
            }
            u64 s = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += weight(x[j], y[j]);
            s = warp_sum(s);
            if (lane == 0) sums[c - c0] = s;
            mine += s;
        }
        __shared__ u64 warp_s[kThreads / 32];
        if (lane == 0) warp_s[warp] = mine;
        __syncthreads();
        mine = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) mine += warp_s[i];
        if (tid == 0) total_s[pass] = mine;
        cluster.sync();
        all = before = 0;
        for (int r = 0; r < C; ++r) {
            const u64 s = *cluster.map_shared_rank(&total_s[pass], r);
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
            w[j] = i < a.V ? weight(p[i], q ? q[i] : 0.f) : 0;
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
    cluster.sync();  // a CTA's totals stay readable until all have read them
}

}  // namespace verify
}  // namespace gdn
