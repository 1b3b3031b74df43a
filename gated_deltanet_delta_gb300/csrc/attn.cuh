// attn.cuh -- what the kernels of attn_paged share: the argument block, the division of the work among
// CTAs, and the joining of partial results.
//
// What is computed.  Sequence n has L = kv_lens[n] cached keys, its m = cu[n+1] - cu[n] new tokens'
// own included; its query i stands at position L - m + i and sees the keys up to that position.  Query
// head hq reads key head hq / G, G = Hq / Hkv:
//     s_j = scale q.k_j,   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = ln sum_j e^{s_j}.
// All kernels make one pass over the keys with a running maximum, in base 2: y_j = s_j log2(e),
// p_j = 2^{y_j - ref}, l = sum p_j and acc = sum p_j v_j in fp32.  ref follows the running maximum only
// when that is more than kRefSlack above it, so p_j <= 2^kRefSlack and the accumulators are rescaled
// a few times per row instead of at every tile; any ref gives the same quotient.
//
// Division of the work.  The G heads that share a key head are rows of one tile: row r of a query tile
// is token i0 + r / G and head h G + r % G, so a key row is read once for all of them.  A unit is
// (sequence, key head, query tile); it costs as many key tiles as its last token sees.  All units'
// key tiles form one list (sequences, then heads, then query tiles, then key tiles), and CTA c takes
// entries [c per, (c+1) per): every CTA has the same work whatever the lengths are, one long sequence
// included.  A unit that spans CTAs leaves one partial (acc, ref, l) per CTA in the workspace (at most
// two per CTA: of the unit that its range begins inside, and of the one that it ends inside), and
// attn_combine_kernel joins them in the order of the keys, so results do not depend on timing.
// The lengths are on the device; every CTA finds its range from them itself.
#pragma once

#include "attn_mma.cuh"
#include "common.cuh"
#include "kernel_args.h"

namespace gdn {
namespace attn {

constexpr float kRefSlack = 8.f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Seq {
    int m, L;       // new tokens, cached keys
    long long q0;   // first query row
};

// Sequence n, with m = 0 (nothing to do) where its bounds are malformed.
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int n, bool* bad) {
    const long long b = a.cu[n], e = a.cu[n + 1], L = a.kv_lens[n];
    Seq s;
    s.q0 = b;
    *bad = b < 0 || e < b || e > a.T || L < 0 || L > static_cast<long long>(a.max_pages) * a.page_size;
    s.m = *bad ? 0 : static_cast<int>(e - b);
    s.L = *bad ? 0 : static_cast<int>(L);
    return s;
}

// Key tiles of query tile qt: what its last token sees, at least one (a tile that sees nothing still
// has to write its zeros).
template <int BN>
__device__ __forceinline__ int unit_tiles(const AttnArgs& a, const Seq& s, int qt) {
    const int last = min((qt + 1) * a.tq, s.m);
    return max(1, (s.L - s.m + last + BN - 1) / BN);
}
template <int BN>
__device__ __forceinline__ long long seq_tiles(const AttnArgs& a, const Seq& s) {
    long long w = 0;
    const int nq = (s.m + a.tq - 1) / a.tq;
    for (int qt = 0; qt < nq; ++qt) w += unit_tiles<BN>(a, s, qt);
    return w;
}

__device__ __forceinline__ long long shfl_up_ll(long long v, int d) {
    return static_cast<long long>(__shfl_up_sync(kFullMask, static_cast<unsigned long long>(v), d));
}

// Position of an entry of the work list.
struct Place {
    int n, h, qt, tile;
    Seq s;
    int nk;  // key tiles of the unit
};

struct PlanSmem {
    long long warp[32];
    long long rem;
    int n;
};

// Total weight of the list: the sum over sequences, times Hkv.  `w0` receives the weight of sequence
// threadIdx.x (the first chunk of locate()).  status bits are set by the CTA with report = true.
template <int BN, int NT>
__device__ __forceinline__ long long plan_total(const AttnArgs& a, PlanSmem& sm, long long& w0, bool report) {
    const int tid = threadIdx.x;
    long long sum = 0;
    w0 = 0;
    for (int n = tid; n < a.num_seqs; n += NT) {
        bool bad;
        const Seq s = load_seq(a, n, &bad);
        if (bad && report) atomicOr(a.status, kStatusBadSeqlens);
        const long long w = seq_tiles<BN>(a, s) * a.Hkv;
        if (n == tid) w0 = w;
        sum += w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += static_cast<long long>(__shfl_xor_sync(kFullMask, static_cast<unsigned long long>(sum), o));
    if ((tid & 31) == 0) sm.warp[tid >> 5] = sum;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) total += sm.warp[i];
    __syncthreads();
    return total;
}

// The place of entry `at` (0 <= at < total).  All threads of the block call it.
template <int BN, int NT>
__device__ __forceinline__ Place locate(const AttnArgs& a, PlanSmem& sm, long long w0, long long at) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    long long base = 0;
    for (int n0 = 0; n0 < a.num_seqs; n0 += NT) {
        long long w = 0;
        if (n0 == 0) {
            w = w0;
        } else if (n0 + tid < a.num_seqs) {
            bool bad;
            const Seq s = load_seq(a, n0 + tid, &bad);
            w = seq_tiles<BN>(a, s) * a.Hkv;
        }
        long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = shfl_up_ll(inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sm.warp[wid] = inc;
        __syncthreads();
        long long before = base, total = base;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            const long long x = sm.warp[i];
            if (i < wid) before += x;
            total += x;
        }
        const long long lo = before + inc - w;
        if (at >= lo && at < lo + w) {
            sm.n = n0 + tid;
            sm.rem = at - lo;
        }
        __syncthreads();
        if (at < total) break;
        base = total;
    }
    Place p;
    p.n = sm.n;
    bool bad;
    p.s = load_seq(a, p.n, &bad);
    const long long per_head = seq_tiles<BN>(a, p.s);
    const long long rem = sm.rem;
    p.h = static_cast<int>(rem / per_head);
    long long r = rem - p.h * per_head;
    p.qt = 0;
    p.nk = unit_tiles<BN>(a, p.s, 0);
    while (r >= p.nk) {
        r -= p.nk;
        p.nk = unit_tiles<BN>(a, p.s, ++p.qt);
    }
    p.tile = static_cast<int>(r);
    return p;
}

// The first entry of the unit after p's (which must exist).
template <int BN>
__device__ __forceinline__ void next_unit(const AttnArgs& a, Place& p) {
    p.tile = 0;
    if ((p.qt + 1) * a.tq < p.s.m) {
        ++p.qt;
    } else {
        p.qt = 0;
        if (++p.h == a.Hkv) {
            p.h = 0;
            bool bad;
            do p.s = load_seq(a, ++p.n, &bad);
            while (p.s.m == 0);
        }
    }
    p.nk = unit_tiles<BN>(a, p.s, p.qt);
}

// pos / page_size for 0 <= pos < 2^31: page_mul = ceil(2^(31 + s) / page_size), 2^s >= page_size.
__device__ __forceinline__ int page_of(const AttnArgs& a, int pos) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(pos)) * a.page_mul) >> a.page_shift);
}

// Element offset (in rows of D) of key `pos` of sequence n, head h; -1 where its page is outside the cache.
__device__ __forceinline__ long long row_of(const AttnArgs& a, int n, int h, int pos) {
    const int pg = page_of(a, pos);
    const long long page = a.table[static_cast<long long>(n) * a.max_pages + pg];
    if (page < 0 || page >= a.num_pages) {
        atomicOr(a.status, kStatusBadCacheIndex);
        return -1;
    }
    return (page * a.Hkv + h) * a.page_size + (pos - pg * a.page_size);
}

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What a CTA leaves for attn_combine_kernel: parts = 0, or the unit that begins in its range and goes on
// in the next parts - 1 CTAs'.
__device__ __forceinline__ void leave_join(const AttnArgs& a, const Place& p, int t0, int t1, long long per) {
    AttnJoin j;
    const int i0 = p.qt * a.tq;
    j.parts = t0 > 0 || t1 == p.nk ? 0 : 1 + static_cast<int>((p.nk - t1 + per - 1) / per);
    j.rows = min(a.tq, p.s.m - i0) * a.G;
    j.h = p.h;
    j.pad = 0;
    j.token = p.s.q0 + i0;
    a.joins[blockIdx.x] = j;
}
__device__ __forceinline__ void leave_no_join(const AttnArgs& a) { a.joins[blockIdx.x].parts = 0; }

// Joins the partials of the unit that begins in CTA blockIdx.x of the main kernel and ends in a later one:
// slot 1 of that CTA and slot 0 of the parts - 1 after it, in that order.  A slot holds R rows of D sums,
// then R references, then R values of l.  D / 4 threads make a group, which owns a row (four columns per
// thread); with more groups than rows, several groups share a row's partials.  blockIdx.y: rows RB ..
constexpr int kCombineThreads = 512;
__device__ __forceinline__ void weigh(float f, float lp, const float4& v, float& l, float4& acc) {
    l = fmaf(f, lp, l);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
}
template <int D>
__global__ void __launch_bounds__(kCombineThreads) attn_combine_kernel(const __grid_constant__ AttnArgs a, int R, int RB) {
    constexpr int TPR = D / 4, GROUPS = kCombineThreads / TPR;
    __shared__ float4 acc_s[kCombineThreads];
    __shared__ float2 rl_s[GROUPS];
    pdl_wait();
    const AttnJoin j = a.joins[blockIdx.x];
    const int r0 = blockIdx.y * RB, nr = min(RB, j.rows - r0);
    if (j.parts < 2 || nr <= 0) return;
    const int g = threadIdx.x / TPR, lane = threadIdx.x % TPR, col = lane * 4;
    const int slices = max(1, min(j.parts, GROUPS / nr));
    const long long slot = static_cast<long long>(R) * (D + 2);
    const float* first = a.part + (blockIdx.x * 2LL + 1) * slot;
    const float* rest = a.part + (blockIdx.x + 1) * 2LL * slot - 2 * slot;  // partial i >= 1 at rest + 2 i slot
    // partials sl, sl + slices, .. of row r
    auto gather = [&](int r, int sl, float& ref, float& l, float4& acc) {
        ref = -INFINITY;
#pragma unroll 8
        for (int i = sl; i < j.parts; i += slices)
            ref = fmaxf(ref, (i == 0 ? first : rest + i * 2 * slot)[static_cast<long long>(R) * D + r]);
        const float base = ref == -INFINITY ? 0.f : ref;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = sl; i < j.parts; i += slices) {
            const float* s = i == 0 ? first : rest + i * 2 * slot;
            const float4 v = *reinterpret_cast<const float4*>(s + static_cast<long long>(r) * D + col);
            weigh(exp2f(s[static_cast<long long>(R) * D + r] - base), s[static_cast<long long>(R) * (D + 1) + r], v, l, acc);
        }
    };
    auto finish = [&](int r, float ref, float l, const float4& acc) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const long long row = (j.token + r / a.G) * a.Hq + j.h * a.G + r % a.G;
        uint2 w;
        w.x = a.f16 ? pack2<true>(acc.x * inv, acc.y * inv) : pack2<false>(acc.x * inv, acc.y * inv);
        w.y = a.f16 ? pack2<true>(acc.z * inv, acc.w * inv) : pack2<false>(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + col) = w;
        if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(l)) * kLn2;
    };
    float ref, l;
    float4 acc;
    if (slices == 1) {
        for (int r = g; r < nr; r += GROUPS) {
            gather(r0 + r, 0, ref, l, acc);
            finish(r0 + r, ref, l, acc);
        }
        return;
    }
    if (g < nr * slices) {
        gather(r0 + g % nr, g / nr, ref, l, acc);
        acc_s[threadIdx.x] = acc;
        if (lane == 0) rl_s[g] = make_float2(ref, l);
    }
    __syncthreads();
    if (g >= nr) return;
    float top = -INFINITY;
    for (int k = 0; k < slices; ++k) top = fmaxf(top, rl_s[k * nr + g].x);
    const float base = top == -INFINITY ? 0.f : top;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < slices; ++k) {
        const float2 rl = rl_s[k * nr + g];
        weigh(exp2f(rl.x - base), rl.y, acc_s[(k * nr + g) * TPR + lane], l, acc);
    }
    finish(r0 + g, top, l, acc);
}

}  // namespace attn
}  // namespace gdn
