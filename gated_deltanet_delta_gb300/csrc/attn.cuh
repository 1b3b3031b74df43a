// attn.cuh -- what the kernels of attn_paged share: the argument block, the division of the work among
// CTAs, and the joining of partial results.
//
// What is computed.  Sequence n has L = kv_lens[n] cached keys, its m = cu[n+1] - cu[n] new tokens'
// own included; its query i stands at position L - m + i and sees the keys up to that position.  Query
// head hq reads key head hq / G, G = Hq / Hkv:
//     s_j = scale q.k_j,   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = ln sum_j e^{s_j}.
// All kernels make one pass over the keys with a running maximum, in base 2: y_j = s_j log2(e),
// p_j = 2^{y_j - ref + kLift}, l = 2^-kLift sum p_j and acc = sum p_j v_j in fp32.  ref follows the running
// maximum only when that is more than kRefSlack above it, so p_j <= 2^(kRefSlack + kLift) and the accumulators are
// rescaled a few times per row instead of at every tile; any ref gives the same quotient.  p_j is rounded to the
// operands' type for the product with v_j.  In binary16 what is below 2^-25 becomes 0, and would count in l but not in
// acc: without the lift 2^17 keys of 2^-26 of the largest weight were missing from the output.  kLift puts p_j at the
// top of binary16's range (at most 2^15), so that only weights below 2^-32 of the largest are lost; n of them are n 2^-32 of
// the output at most, less than binary16's own rounding up to 2^20 keys.
//
// Division of the work.  The G heads that share a key head are rows of one tile: row r of a query tile
// is token i0 + r / G and head h G + r % G, so a key row is read once for all of them.  A unit is
// (sequence, key head, query tile); it takes as many key tiles as its last token sees.  Its cost, counted
// in products of 128 (16) rows with a key tile, is wt per key tile (2 where it has two row tiles) plus ov for
// starting and ending it.  All units' costs form one line (sequences, then heads, then query tiles), and
// CTA c takes the stretch [c per, (c+1) per): every CTA has the same cost whatever the lengths are, one
// long sequence included.  (The time differs by what the cost leaves out, ends and joins: the longest SM was at work
// 6 % longer than the mean in 16-bit single tokens, 9 % in prompts of 64-wide heads, 17 % in 8-bit chunks, 28 % in
// 8-bit windows of 256-wide heads.)  A stretch's end inside a unit cuts it between two key tiles.  A unit that spans
// CTAs leaves one partial (acc, ref, l) per CTA in the workspace (at most two per CTA: of the unit that its
// stretch begins inside, and of the one that it ends inside), and attn_combine_kernel joins them in the
// order of the keys, so results do not depend on timing.  The lengths are on the device; every CTA finds
// its stretch from them itself.
#pragma once

#include "attn_mma.cuh"
#include "common.cuh"
#include "kernel_args.h"

namespace gdn {
namespace attn {

constexpr float kRefSlack = 8.f, kLift = 7.f, kUnlift = 1.f / 128;  // kUnlift = 2^-kLift
constexpr uint32_t kWaitPolls = 1u << 22;  // the built-in limit of a wait (seconds), and that of the waits after one gave up
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
    // (one limit, the least of the two, in the arguments: heads of 256 5 % slower, for its registers)
    *bad = b < 0 || e < b || e > a.T || L < 0 || L > static_cast<long long>(a.max_pages) * a.page_size || L > kAttnMaxKeys;
    s.m = *bad ? 0 : static_cast<int>(e - b);
    s.L = *bad ? 0 : static_cast<int>(L);
    return s;
}

// a / b for a >= 0, b > 0: 64-bit division takes some hundred cycles, 32-bit a few tens.
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (static_cast<unsigned long long>(a | b) >> 32) return a / b;
    return static_cast<unsigned>(a) / static_cast<unsigned>(b);
}

// How a kernel tiles: BN keys, SL row tiles of ROWS rows per unit.
template <int BN_, int SL_, int ROWS_>
struct Tiling {
    static constexpr int BN = BN_, SL = SL_, ROWS = ROWS_;
};

// sum_{i < n} floor((a i + b) / m), all not negative: the steps of Euclid's algorithm (lattice points
// under a line).
__device__ __forceinline__ long long floor_sum(long long n, unsigned m, unsigned a, unsigned b) {
    long long sum = 0;
    while (n > 0) {
        sum += (n - 1) * n / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const unsigned long long top = static_cast<unsigned long long>(a) * n + b;
        if (top < m) break;
        n = divide(static_cast<long long>(top), m);
        b = static_cast<unsigned>(top - static_cast<unsigned long long>(n) * m);
        const unsigned x = m;
        m = a;
        a = x;
    }
    return sum;
}

// Key tiles of query tile qt: what its last token sees, at least one (a tile that sees nothing still
// has to write its zeros).
template <class T>
__device__ __forceinline__ int unit_tiles(const AttnArgs& a, const Seq& s, int qt) {
    const int last = min((qt + 1) * a.tq, s.m);
    return max(1, (s.L - s.m + last + T::BN - 1) / T::BN);
}
// Cost per key tile of query tile qt.
template <class T>
__device__ __forceinline__ int unit_wt(const AttnArgs& a, const Seq& s, int qt) {
    return T::SL == 2 && min(a.tq, s.m - qt * a.tq) * a.G > T::ROWS ? 2 : 1;
}
// Cost of query tiles 0 .. k - 1, none of them the sequence's last.
template <class T>
__device__ __forceinline__ long long cost_before(const AttnArgs& a, const Seq& s, int k) {
    if (k == 0) return 0;
    // tile i's last token sees base + (i + 1) tq keys; the first `ones` of them at most one tile
    const int base = s.L - s.m;
    const int ones = min(k, max(0, T::BN - base) / a.tq);
    const long long tiles = ones + floor_sum(k - ones, T::BN, a.tq, base + (ones + 1) * a.tq + T::BN - 1);
    return tiles * unit_wt<T>(a, s, 0) + static_cast<long long>(k) * a.ov;
}
template <class T>
__device__ __forceinline__ long long seq_cost(const AttnArgs& a, const Seq& s) {
    if (s.m == 0) return 0;
    const int last = (s.m - 1) / a.tq;
    return cost_before<T>(a, s, last) + unit_tiles<T>(a, s, last) * unit_wt<T>(a, s, last) + a.ov;
}

__device__ __forceinline__ long long shfl_up_ll(long long v, int d) {
    return static_cast<long long>(__shfl_up_sync(kFullMask, static_cast<unsigned long long>(v), d));
}

struct PlanSmem {
    long long warp[32];
    long long rem;
    int n;
};

// A CTA's walk along its stretch: the unit it is in, and the unit's key tiles t0 .. t1 - 1 that are its.
struct Walk {
    int n, h, qt;
    Seq s;
    int nk, wt;            // the unit's key tiles and their cost
    int t0, t1;
    long long begin, end;  // the unit's begin; the stretch's end
};

__device__ __forceinline__ int cut(const AttnArgs& a, const Walk& w, long long at) {  // key tiles before `at`
    const long long x = at - w.begin - a.ov;
    return x <= 0 ? 0 : static_cast<int>(min(static_cast<long long>(w.nk), (x + w.wt - 1) >> (w.wt - 1)));  // wt: 1 or 2
}
template <class T>
__device__ __forceinline__ void enter(const AttnArgs& a, Walk& w, long long from) {
    w.nk = unit_tiles<T>(a, w.s, w.qt);
    w.wt = unit_wt<T>(a, w.s, w.qt);
    w.t0 = cut(a, w, from);
    w.t1 = cut(a, w, w.end);
}
// On to the next unit that has tiles for this CTA; false at the stretch's end.
template <class T>
__device__ __forceinline__ bool advance(const AttnArgs& a, Walk& w) {
    do {
        const long long past = w.begin + static_cast<long long>(w.nk) * w.wt + a.ov;
        if (w.end <= past) return false;
        w.begin = past;
        if ((w.qt + 1) * a.tq < w.s.m) {
            ++w.qt;
        } else {
            w.qt = 0;
            if (++w.h == a.Hkv) {
                w.h = 0;
                bool bad;
                do w.s = load_seq(a, ++w.n, &bad);
                while (w.s.m == 0);
            }
        }
        enter<T>(a, w, w.begin);
    } while (w.t0 >= w.t1);
    return true;
}

// This CTA's stretch and its first unit; false where it has no work.  All threads of the block call it.
// status bits are set by CTA 0.
template <class T, int NT>
__device__ __forceinline__ bool plan(const AttnArgs& a, PlanSmem& sm, Walk& w, long long& per) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    long long sum = 0, first = 0;  // costs of this thread's sequences; of the first one
    for (int n = tid; n < a.num_seqs; n += NT) {
        bool bad;
        const Seq s = load_seq(a, n, &bad);
        if (bad && blockIdx.x == 0) atomicOr(a.status, kStatusBadSeqlens);
        const long long c = seq_cost<T>(a, s) * a.Hkv;
        if (n == tid) first = c;
        sum += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += static_cast<long long>(__shfl_xor_sync(kFullMask, static_cast<unsigned long long>(sum), o));
    if (lane == 0) sm.warp[wid] = sum;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) total += sm.warp[i];
    per = max(divide(total + gridDim.x - 1, gridDim.x), static_cast<long long>(a.min_per));
    const long long at = blockIdx.x * per;
    if (at >= total) return false;
    // the sequence that `at` falls in
    long long base = 0;
    for (int n0 = 0; n0 < a.num_seqs; n0 += NT) {
        long long c = first;
        if (n0 > 0) {
            c = 0;
            if (n0 + tid < a.num_seqs) {
                bool bad;
                const Seq s = load_seq(a, n0 + tid, &bad);
                c = seq_cost<T>(a, s) * a.Hkv;
            }
        }
        long long inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = shfl_up_ll(inc, o);
            if (lane >= o) inc += u;
        }
        __syncthreads();  // sm.warp has been read
        if (lane == 31) sm.warp[wid] = inc;
        __syncthreads();
        long long before = base, all = base;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            const long long x = sm.warp[i];
            if (i < wid) before += x;
            all += x;
        }
        const long long lo = before + inc - c;
        if (at >= lo && at < lo + c) {
            sm.n = n0 + tid;
            sm.rem = at - lo;
        }
        if (at < all) break;
        base = all;
    }
    __syncthreads();
    w.n = sm.n;
    w.end = min(at + per, total);
    bool bad;
    w.s = load_seq(a, w.n, &bad);
    const long long rem = sm.rem, head = seq_cost<T>(a, w.s);
    w.h = static_cast<int>(divide(rem, head));
    const long long r = rem - w.h * head;
    // the last query tile that begins at or before r: costs rise, so count the tiles that do
    const int tiles = (w.s.m + a.tq - 1) / a.tq;
    int count = 0;
    for (int q0 = 0; q0 < tiles; q0 += NT) {
        const int c = __syncthreads_count(q0 + tid < tiles && cost_before<T>(a, w.s, q0 + tid) <= r);
        count += c;
        if (c < NT) break;
    }
    w.qt = count - 1;
    w.begin = at - (r - cost_before<T>(a, w.s, w.qt));
    enter<T>(a, w, at);
    return w.t0 < w.t1 || advance<T>(a, w);
}

// pos / page_size for 0 <= pos < 2^31: page_mul = ceil(2^(31 + s) / page_size), 2^s >= page_size.
__device__ __forceinline__ int page_of(const AttnArgs& a, int pos) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(pos)) * a.page_mul) >> a.page_shift);
}

// The page table's entry for key `pos` of sequence n.  Looked at (row_of) only when it is needed: a check
// right behind the load would wait for it.
__device__ __forceinline__ long long page_entry(const AttnArgs& a, int n, int pos) {
    return a.table[static_cast<long long>(n) * a.max_pages + page_of(a, pos)];
}
// Offset (in rows of D) of key `pos` of head h, which is in page `page`; -1 where that is outside the cache.
__device__ __forceinline__ long long row_of(const AttnArgs& a, long long page, int h, int pos) {
    if (page < 0 || page >= a.num_pages) {
        atomicOr(a.status, kStatusBadCacheIndex);
        return -1;
    }
    return (page * a.Hkv + h) * a.page_size + (pos - page_of(a, pos) * a.page_size);
}

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What a CTA leaves for attn_combine_kernel: parts = 0, or the unit that begins in its stretch and goes on
// in the next parts - 1 CTAs' (those whose stretch begins before the unit's last key tile).
__device__ __forceinline__ void leave_join(const AttnArgs& a, const Walk& w, long long per) {
    AttnJoin j;
    const int i0 = w.qt * a.tq;
    j.parts = 0;
    if (w.t0 == 0 && w.t1 < w.nk)
        j.parts = 1 + static_cast<int>(divide(w.begin + a.ov + static_cast<long long>(w.nk - 1) * w.wt, per) - blockIdx.x);
    j.rows = min(a.tq, w.s.m - i0) * a.G;
    j.h = w.h;
    j.pad = 0;
    j.token = w.s.q0 + i0;
    a.joins[blockIdx.x] = j;
}
__device__ __forceinline__ void leave_no_join(const AttnArgs& a) { a.joins[blockIdx.x].parts = 0; }

// Joins the partials of the unit that begins in CTA blockIdx.x of the main kernel and ends in a later one:
// slot 1 of that CTA and slot 0 of the parts - 1 after it, in that order.  A slot holds R rows of D sums,
// then R references, then R values of l.  D / 4 threads make a group, which owns a row (four columns per
// thread); with more groups than rows, several groups share a row's partials.  blockIdx.y: rows RB ..
constexpr int kCombineThreads = 256;
__device__ __forceinline__ void weigh(float f, float lp, const float4& v, float& l, float4& acc) {
    l = fmaf(f, lp, l);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
}
template <int D>
__global__ void __launch_bounds__(kCombineThreads, 5) attn_combine_kernel(const __grid_constant__ AttnArgs a, int R, int RB) {
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
    // partials sl, sl + slices, .. of row r, three at a time (their loads in flight together)
    auto gather = [&](int r, int sl, float& ref, float& l, float4& acc) {
        ref = -INFINITY;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = sl; i0 < j.parts; i0 += 3 * slices) {
            float rf[3], lp[3];
            float4 v[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int i = i0 + k * slices;
                const float* s = i == 0 ? first : rest + i * 2 * slot;
                const bool on = i < j.parts;
                rf[k] = on ? s[static_cast<long long>(R) * D + r] : -INFINITY;
                lp[k] = on ? s[static_cast<long long>(R) * (D + 1) + r] : 0.f;
                v[k] = on ? *reinterpret_cast<const float4*>(s + static_cast<long long>(r) * D + col) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const float top = fmaxf(fmaxf(rf[0], rf[1]), fmaxf(rf[2], ref));
            const float base = top == -INFINITY ? 0.f : top, f = exp2f(ref - base);
            l *= f;
            acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
            for (int k = 0; k < 3; ++k) weigh(exp2f(rf[k] - base), lp[k], v[k], l, acc);
            ref = top;
        }
    };
    auto finish = [&](int r, float ref, float l, const float4& acc) {
        const float inv = l > 0.f || l != l ? kUnlift / l : 0.f;
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
