// attn_tiles.cuh -- attn_paged for many query rows per key head (drafted windows, chunks, prompts): tiles
// of 128 rows on the tensor cores (tcgen05, accumulators in TMEM).
//
// Per key tile of BN keys and 128 rows:  S = Q K^T (128 x BN x D),  P = 2^{y - ref + kLift},  O += P V
// (128 x D x BN).  S, P (over S's columns) and O live in TMEM; Q, K and V tiles in shared memory in the
// 128-byte-swizzled operand layouts; a row's reference and sum in its thread's registers.
// Two S buffers keep the tensor core busy while one of them is exponentiated.  D <= 128: a unit has up to
// 256 rows, two row tiles ("slots") with an accumulator each that share every K and V tile; a unit of at
// most 128 rows uses the slots for alternate key tiles, and the two accumulators are added at its end.
// D = 256: one row tile and one accumulator (256 columns), key tiles of 64 in two S buffers.
// So operation s (s = 0, 1, ..) works in buffer s & 1 on key tile s / 2 (two row tiles) or s.
//
// Roles, 512 threads: warpgroups 0 and 1 are the softmax, one per buffer (D = 256: warpgroup 0 has both; thread i
// owns TMEM lane i, a row); warpgroup 2 loads; one lane of warp 12 issues every MMA:
//   S(0) S(1) | P(0)? PV(0) S(2) | P(1)? PV(1) S(3) ..
// Operations of one issuing thread run in order, so S(s + 2) overwrites a buffer only after PV(s) has
// read P from it.  D = 128: P is handed over in two halves, so that its products begin while the second half is
// exponentiated: the chain S, softmax, PV of a slot is what bounds long chunks.  D = 64 has TMEM left for P
// besides S, so there S(s + 2) is issued as soon as S(s) has been read, the softmax never waits for it, and a
// hand-over in halves only costs (prompts 264 us, without it 261).
// The loader gathers rows by page: whole boxes of rows by TMA, the ragged end of the keys by cp.async with
// zero fill (nothing stale may meet a weight of zero).
// 8-bit caches: warp 13 (D = 256: 13 the keys, 14 the values) copies into a staging ring, warp 15 fetches the
// scales, and warpgroup 2 (D = 256: 2 the keys, 1 the values) does nothing but widen into the tiles, 128 threads
// on 2-clock conversions; one warpgroup that did all three took 136 us where this took 111 (the windows below).
// attn_rows.cuh says how the scales are applied.
//
// Measured: chunks of 4096 tokens over up to 15360 keys, two sequences, 32 / 8 heads of 128: 910 to 925 us, 1.4
// PFLOP/s, bound by the chain above; whole prompts of up to 4096 tokens, nine, 16 / 4 heads of 64: 262 to 271 us, where no
// unit is the limit (exponentials and tensor core 25 % each, issue 40 %) but the latency of two softmax warps per
// scheduler, and the SMs' uneven ends; windows of 8 tokens over up to 15360 8-bit keys, 32, 16 / 2 heads of 256: 113
// us, bound by the softmax of one warpgroup, and by uneven ends.
//
// Every wait is bounded: one that runs out sets GDN_STATUS_TIMEOUT and the CTA's limit of polls to 0, on which
// all roles leave; copies and MMAs in flight are waited for (bounded) before the CTA ends.
#pragma once

#include "attn.cuh"
#include "attn_mma.cuh"
#include "tcgen05.cuh"

namespace gdn {
namespace attn {

constexpr int kTilesNT = 512;

template <int D, bool F8>
struct TilesCfg {
    static constexpr int BN = D == 256 ? 64 : 128;         // keys per tile
    static constexpr int SLOTS = D == 256 ? 1 : 2;         // row tiles per unit
    static constexpr int R = 128 * SLOTS;                  // rows per unit
    static constexpr bool QTM = D == 256;                  // queries in TMEM, not in shared memory
    static constexpr bool PSEP = D == 64;                  // P in columns of its own, not over S
    static constexpr bool HALF = SLOTS == 2 && !PSEP;      // P handed over in halves
    static constexpr bool DUAL = F8 && D == 256;           // warpgroup 1, idle else, widens the values
    static constexpr uint32_t QTILE = 128u * D * 2, TILE = static_cast<uint32_t>(BN) * D * 2;
    static constexpr uint32_t RAW = F8 ? TILE / 2 : 0;
    // K and V tiles in shared memory.  Two widening warpgroups: 4, so that each has places of its own.
    static constexpr int NST = F8 ? (DUAL ? 4 : (PSEP ? 5 : 3)) : (D == 64 ? 8 : (D == 128 ? 5 : 6));
    // copy groups in flight behind the newest: at most NST - 2 (PSEP: NST - 5), as S(s + 2) needs its K tile
    // before the V tile (the two V tiles and a K tile) before it is released
    static constexpr int LAG = 3;
    // 8 bits: staging slots, one ring for all tiles or (DUAL) one for the keys' and one for the values'
    static constexpr int NRAW = F8 ? (D == 64 ? 6 : (DUAL ? 2 : 3)) : 0, RINGS = (DUAL ? 2 : 1) * NRAW;
    static constexpr uint32_t SCN = 4;                     // tiles whose keys' scales are held
    static constexpr int BOX = BN / 4;                     // most rows of one TMA box: a loader warp's rows
    static constexpr uint32_t OFF_KV = QTM ? 0 : SLOTS * QTILE;
    static constexpr uint32_t OFF_RAW = OFF_KV + NST * TILE;
    static constexpr uint32_t OFF_SC = OFF_RAW + RINGS * RAW;             // ks, log2 vs, 1 / vs of SCN tiles
    static constexpr uint32_t OFF_RS = OFF_SC + (F8 ? SCN * 3u * BN * 4 : 0);  // row scales of two units
    static constexpr uint32_t USED = OFF_RS + (F8 && !QTM ? 2 * R * 4 : 0);
    static constexpr uint32_t SMEM = USED + 1024;          // 1024-byte alignment
    static constexpr uint32_t TM_S = 0, TM_Q = 128, TM_O = 256, TM_SB = BN;  // TMEM columns
    static constexpr uint32_t TM_P = PSEP ? 384 : TM_S, TM_PB = PSEP ? 64 : TM_SB;
};

// Barriers: queries full / empty, S, P (halves first), products with V done, accumulators read, (ref, l)
// handed over / read, end; then KV_FULL and KV_EMPTY of every place and, for 8 bits, staging slots and scales
// full / empty.
enum : int {
    TB_QF = 0, TB_QE, TB_S0, TB_S1, TB_P0, TB_P1, TB_H0, TB_H1, TB_R0, TB_R1, TB_OD0, TB_OD1, TB_OF0, TB_OF1, TB_MF, TB_ME, TB_DRAIN, TB_KV
};

__device__ __forceinline__ void tm_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Pairs of fp32 operations in one instruction (f32x2).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 p, float* x) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x[0]), "=f"(x[1]) : "l"(p)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// x <- 2^(x times + plus), both elements
__device__ __forceinline__ void pair_exp2(float* x, float times, float plus) {
    unpair(fma2(pair(x[0], x[1]), pair(times, times), pair(plus, plus)), x);
    x[0] = fast_exp2(x[0]);
    x[1] = fast_exp2(x[1]);
}
// y <- x (c k) + v.  In this order, because c (the softmax scale over the query row's power of two) and k (the key's
// scale) may be as large and as small as numbers get, and only their product is sure not to be.
__device__ __forceinline__ void pair_fma(float* y, const float* x, float c, float k0, float k1, float v0, float v1) {
    unpair(fma2(pair(x[0], x[1]), mul2(pair(c, c), pair(k0, k1)), pair(v0, v1)), y);
}
__device__ __forceinline__ void pair_add(float* s, const float* x) { unpair(add2(pair(s[0], s[1]), pair(x[0], x[1])), s); }
__device__ __forceinline__ void pair_mac(float* s, const float* x, float k0, float k1) {
    unpair(fma2(pair(x[0], x[1]), pair(k0, k1), pair(s[0], s[1])), s);
}

// The same value in every lane, as the compiler sees it too.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFullMask, x, 0); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return static_cast<uint64_t>(uniform(static_cast<uint32_t>(x >> 32))) << 32 | uniform(static_cast<uint32_t>(x));
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(one));
    return one != 0;
}

// Registers per thread after the roles part: the softmax holds a row of S (the launch's 512 x 128 registers
// are 128 x (184 + 184 + 72 + 72)).
constexpr int kRegsLaunch = 128, kRegsSoftmax = 184, kRegsOther = 72;
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int D, bool F16, bool F8>
__global__ void __launch_bounds__(kTilesNT, 1) attn_tiles_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using C = TilesCfg<D, F8>;
    constexpr bool MF16 = F16 || F8;
    constexpr int BN = C::BN, NST = C::NST, LAG = C::LAG, SLOTS = C::SLOTS;
    (void)LAG;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanSmem plan_s;
    constexpr int KV_FULL = TB_KV, KV_EMPTY = TB_KV + NST, RAW_FULL = TB_KV + 2 * NST, RAW_EMPTY = RAW_FULL + C::RINGS,
                  SC_FULL = RAW_EMPTY + C::RINGS, SC_EMPTY = SC_FULL + (F8 ? C::SCN : 0), NBAR = SC_EMPTY + (F8 ? C::SCN : 0);
    __shared__ uint64_t bars[NBAR];
    __shared__ float ml_s[128][2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t most_polls;  // of a wait; 0 once one has run out, so that the others give up
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = tid >> 7;

    typedef Tiling<BN, SLOTS, 128> T;
    Walk p;
    long long per;
    const bool busy = plan<T, kTilesNT>(a, plan_s, p, per);
    pdl_launch();
    if (!busy) {
        if (tid == 256) leave_no_join(a);
        return;
    }

    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    if (warp == 12) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            const bool by_warps = i == TB_QF || (i >= TB_P0 && i <= TB_R1) || i == TB_OF0 || i == TB_OF1 || i == TB_MF ||
                                  i == TB_ME || (i >= KV_FULL && i < KV_EMPTY) || (i >= RAW_EMPTY && i < SC_FULL);
            // TB_QE, 8 bits: the last product with the queries, and each softmax warp that has read its rows' scales
            tc::mbar_init(&bars[i], i == TB_QE && F8 && !C::QTM ? 1 + 4 * SLOTS : (by_warps ? 4 : 1));
        }
        most_polls = a.polls;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot;

    auto wait = [&](int i, uint32_t parity) -> bool {
        // The limit is looked at with the flag, where a wait lasts: a variable bound of the loop took 4 % to 10 % more time
        // (chunk 920 -> 1018 us, prompts 264 -> 281), in every wait's first poll.
        if (tc::mbar_wait_most<kWaitPolls>(&bars[i], parity, &most_polls)) return true;
        most_polls = 0;
        return false;
    };
    auto warp_wait = [&](int i, uint32_t parity) -> bool {
        const bool ok = __all_sync(kFullMask, wait(i, parity));
        tc::fence_after();
        return ok;
    };
    auto one_wait = [&](int i, uint32_t parity) -> bool {
        const bool ok = wait(i, parity);
        tc::fence_after();
        return ok;
    };
    // one arrival for the warp, after all of its lanes' writes
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[i]);
    };

    constexpr int RW = BN / 4;                  // rows of a tile that a loader (widening) warp handles
    constexpr int CHR = (F8 ? D : 2 * D) / 16;  // 16-byte chunks per cached row
    constexpr int PER = RW * CHR / 32;          // chunks per lane and tile
    if (F8 && (wg == 2 || (C::DUAL && wg == 1))) {
        // ------------------------------------------------------------ 8 bits: queries, and widening
        // Tiles are numbered K 0, V 1, K 2, ..; a warpgroup has all of them, or (DUAL) the even or the odd ones.
        regs_down<kRegsOther>();
        const int tl = tid & 127, r0 = (warp & 3) * RW;
        const uint32_t lg = C::DUAL && wg == 1 ? 1 : 0;
        constexpr uint32_t STEP = C::DUAL ? 2 : 1;
        uint32_t stage = lg, par = 1, slot = 0, rpar = 0, unit = 0;  // the next place and its parity, the next staging slot
        bool ok = true;
        if (tid == 256) leave_no_join(a);  // stands if this CTA gives up
        // Lanes 0 .. 3 of every eight take chunks of one row, 4 .. 7 the other half's of the next row: so eight lanes'
        // 16-byte loads, and each of their two stores, fall on different banks.
        const int sub = lane >> 2 & 1, q8 = lane >> 3;
        int rl, cl;  // row within a pass over 32 chunks, and chunk
        if constexpr (CHR == 16) rl = sub, cl = (lane & 3) + 4 * (q8 ^ sub);
        else if constexpr (CHR == 8) rl = 2 * (q8 >> 1) + sub, cl = (lane & 3) + 4 * ((q8 & 1) ^ sub);
        else rl = lane >> 2, cl = lane & 3;
        constexpr int RP = 32 / CHR;  // rows per pass
        for (;;) {
            if constexpr (!C::QTM) {
                const int i0 = p.qt * a.tq, rows = min(a.tq, p.s.m - i0) * a.G;
                ok = warp_wait(TB_QE, (unit & 1) ^ 1);
                if (!ok) break;
                for (int r = tl; r < (rows > 128 ? 256 : 128); r += 128) {
                    const bool on = r < rows;
                    const int tok = on ? r / a.G : 0;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        a.q + (p.s.q0 + i0 + tok) * a.q_stride + static_cast<long long>(p.h * a.G + (on ? r - tok * a.G : 0)) * D);
                    float mx = 0.f;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 w = on ? src[c] : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2<F16>(x[j]);
                            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                    const float up = row_up(mx);
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 w = on ? src[c] : make_uint4(0, 0, 0, 0);
                        uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2<F16>(x[j]);
                            x[j] = pack2<true>(f.x * up, f.y * up);
                        }
                        sts128(sb + (r >> 7) * C::QTILE + tc::sw_chunk(r & 127, c, 128), make_uint4(x[0], x[1], x[2], x[3]));
                    }
                    reinterpret_cast<float*>(sm + C::OFF_RS)[(unit & 1) * C::R + r] = a.scale_log2 * (1.f / up);
                }
                tc::fence_proxy_async();
                warp_arrive(TB_QF);
            }
            const int items = (p.t1 - p.t0) * (C::DUAL ? 1 : 2);
            for (int i = 0; i < items && ok; ++i) {
                const uint32_t ring = lg * C::NRAW + slot;
                ok = warp_wait(RAW_FULL + ring, rpar) && warp_wait(KV_EMPTY + stage, par);
                if (!ok) break;
                const uint32_t raw = sb + C::OFF_RAW + ring * C::RAW + (r0 + rl) * D + cl * 16;
                const uint32_t dst = sb + C::OFF_KV + stage * C::TILE;
                uint4 held[PER];
#pragma unroll
                for (int k = 0; k < PER; ++k) held[k] = lds128(raw + k * (RP * D));
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const int r = r0 + k * RP + rl;
                    const uint4 w = held[k];
                    sts128(dst + tc::sw_chunk(r, 2 * cl, BN), make_uint4(e4m3_lo(w.x), e4m3_hi(w.x), e4m3_lo(w.y), e4m3_hi(w.y)));
                    sts128(dst + tc::sw_chunk(r, 2 * cl + 1, BN), make_uint4(e4m3_lo(w.z), e4m3_hi(w.z), e4m3_lo(w.w), e4m3_hi(w.w)));
                }
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bars[KV_FULL + stage]);
                    tc::mbar_arrive(&bars[RAW_EMPTY + ring]);
                }
                stage += STEP;
                if (stage >= NST) stage -= NST, par ^= 1;
                if (++slot == C::NRAW) slot = 0, rpar ^= 1;
            }
            if (!ok) break;
            ++unit;
            if (tid == 256) leave_join(a, p, per);  // the last unit's stands
            if (!advance<T>(a, p)) break;
        }
    } else if (!F8 && wg == 2) {
        // ------------------------------------------------------------ 16 bits: loader
        // warp w moves rows w RW .. w RW + RW - 1 of every tile; lane l holds the cache offset of one of them
        regs_down<kRegsOther>();
        const int tl = tid & 127, r0 = (warp & 3) * RW, mine = r0 + lane % RW;
        // rows that lie within the keys come by TMA, in boxes of a.box rows that never straddle a page; a
        // warp with a row past the keys (or a page size without a factor of 8) uses cp.async and zero-fills
        const int box = a.box, boxes = box ? RW / box : 0;
        uint32_t open = 0, stage = 0, par = 1, pend = 0, unit = 0;
        bool ok = true;
        if (tid == 256) leave_no_join(a);  // stands if this CTA gives up
        auto finish = [&](uint32_t what) {  // the oldest copy group has landed
            tc::fence_proxy_async();
            warp_arrive(what);
        };
        auto push = [&](uint32_t what) {  // closes a copy group, which fills what barrier `what` stands for
            cp_async_commit();
            pend = pend << 8 | what;
            if (open == LAG) {
                cp_async_wait<LAG>();
                finish(pend >> (8 * LAG) & 0xff);
            } else {
                ++open;
            }
        };
        auto flush = [&]() {
            cp_async_wait<0>();
            for (; open > 0; --open) finish(pend >> (8 * (open - 1)) & 0xff);
        };
        for (;;) {
            const int t0 = p.t0, t1 = p.t1;
            const int i0 = p.qt * a.tq, ntok = min(a.tq, p.s.m - i0), rows = ntok * a.G;
            const int kend = min(t1 * BN, p.s.L - p.s.m + i0 + ntok);
            // ---- queries
            if constexpr (!C::QTM) {
                const int qrows = rows > 128 ? 256 : 128;
                ok = warp_wait(TB_QE, (unit & 1) ^ 1);
                if (!ok) break;
                for (int idx = tl; idx < qrows * (D / 8); idx += 128) {
                    const int r = idx / (D / 8), c = idx % (D / 8);
                    const bool on = r < rows;
                    const int tok = on ? r / a.G : 0;
                    const uint16_t* src = a.q + (p.s.q0 + i0 + tok) * a.q_stride +
                                          static_cast<long long>(p.h * a.G + (on ? r - tok * a.G : 0)) * D + c * 8;
                    cp_async16(sb + (r >> 7) * C::QTILE + tc::sw_chunk(r & 127, c, 128), src, on);
                }
                push(TB_QF);
            }
            // ---- keys and values, tile by tile
            auto entry = [&](int t) -> long long {  // a tile ahead: the page table is some hundred cycles away
                const int pos = t * BN + mine;
                return t < t1 && pos < kend ? page_entry(a, p.n, pos) : 0;
            };
            long long next = entry(t0);
            for (int t = t0; t < t1 && ok; ++t) {
                const int pos = t * BN + mine;
                const long long off = pos < kend ? row_of(a, next, p.h, pos) : -1;
                next = entry(t + 1);
                const bool tma = box && __all_sync(kFullMask, off >= 0);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = warp_wait(KV_EMPTY + stage, par);
                    if (!ok) break;
                    const uint32_t dst = sb + C::OFF_KV + stage * C::TILE;
                    if (tma) {
                        constexpr int COLS = D / 64;  // boxes side by side
                        uint64_t* bar = &bars[KV_FULL + stage];
                        if (lane == 0) tc::mbar_expect_tx(bar, RW * CHR * 16);
                        __syncwarp();
                        for (int i = lane; i < (boxes * COLS + 31) / 32 * 32; i += 32) {
                            const int rb = i / COLS * box, x = i % COLS;
                            const long long ro = __shfl_sync(kFullMask, off, rb % RW);
                            if (i < boxes * COLS)
                                tma_load_2d(dst + x * (BN * 128) + (r0 + rb) * 128, kv ? &maps.v : &maps.k, x * 64, static_cast<int>(ro), bar);
                        }
                    } else {
                        const uint8_t* base = static_cast<const uint8_t*>(kv ? a.vc : a.kc);
#pragma unroll 4
                        for (int i = 0; i < PER; ++i) {
                            const int idx = i * 32 + lane, rl = idx / CHR, c = idx % CHR;
                            const long long ro = __shfl_sync(kFullMask, off, rl);
                            const uint8_t* src = base + (ro < 0 ? 0 : ro * (CHR * 16)) + c * 16;
                            cp_async16(dst + tc::sw_chunk(r0 + rl, c, BN), src, ro >= 0);
                        }
                        push(KV_FULL + stage);
                        // A tile that went this way is handed over at once where the next ones may go by TMA (a page outside
                        // the cache, amid good ones): those push nothing, and wait for places that only this tile's
                        // products free.
                        if (box && kv == 1) flush();
                    }
                    if (++stage == NST) stage = 0, par ^= 1;
                }
                // the queries, copied meanwhile, are handed over behind two tiles' copies
                if (!C::QTM && box && t == t0 + 1 && ok) flush();
            }
            if (!ok) break;
            flush();  // the MMAs of this unit, which free the query tiles, need all of its keys
            ++unit;
            if (tid == 256) leave_join(a, p, per);  // the last unit's stands
            if (!advance<T>(a, p)) break;
        }
        cp_async_wait<0>();
        if (!ok) {  // gave up: leave what TMA copies are in flight (microseconds) a millisecond
            for (int i = 0; i < 100; ++i) __nanosleep(10000);
        }
    } else if (wg == 3) {
        regs_down<kRegsOther>();  // by the whole warpgroup, then its warps part
        if (F8 && (warp == 13 || (C::DUAL && warp == 14))) {
            // ------------------------------------------------------------ 8 bits: copies into the staging ring
            const uint32_t lg = C::DUAL && warp == 14 ? 1 : 0;
            const int box = a.box, boxes = box ? BN / box : 0, mine = lane * box;  // lane i copies box i
            uint32_t slot = 0, par = 1;
            bool ok = true;
            for (;;) {
                const int t0 = p.t0, t1 = p.t1, i0 = p.qt * a.tq, ntok = min(a.tq, p.s.m - i0);
                const int kend = min(t1 * BN, p.s.L - p.s.m + i0 + ntok);
                auto entry = [&](int t) -> long long {  // a tile ahead: the page table is some hundred cycles away
                    const int pos = t * BN + mine;
                    return t < t1 && lane < boxes && pos < kend ? page_entry(a, p.n, pos) : 0;
                };
                long long next = entry(t0);
                for (int t = t0; t < t1 && ok; ++t) {
                    const int pos = t * BN + mine;
                    // boxes whose rows are all keys; the ragged end's rows go one by one
                    const long long off = lane < boxes && pos + box <= kend ? row_of(a, next, p.h, pos) : -1;
                    next = entry(t + 1);
                    const unsigned on = __ballot_sync(kFullMask, off >= 0);
    #pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (C::DUAL && kv != static_cast<int>(lg)) continue;
                        const uint32_t ring = lg * C::NRAW + slot, dst = sb + C::OFF_RAW + ring * C::RAW;
                        ok = warp_wait(RAW_EMPTY + ring, par);
                        if (!ok) break;
                        uint64_t* bar = &bars[RAW_FULL + ring];
                        if (off >= 0) tma_load_2d(dst + mine * D, kv ? &maps.v : &maps.k, 0, static_cast<int>(off), bar);
                        if (__popc(on) * box < BN) {
                            const uint8_t* base = static_cast<const uint8_t*>(kv ? a.vc : a.kc);
                            for (int idx = lane; idx < BN * CHR; idx += 32) {
                                const int r = idx / CHR, c = idx % CHR;
                                if (box && (on >> (r / box) & 1)) continue;
                                const int at = t * BN + r;
                                const long long ro = at < kend ? row_of(a, page_entry(a, p.n, at), p.h, at) : -1;
                                cp_async16(dst + idx * 16, base + (ro < 0 ? 0 : ro * D) + c * 16, ro >= 0);
                            }
                            cp_async_commit();
                            cp_async_wait<0>();
                        }
                        __syncwarp();
                        if (lane == 0) tc::mbar_expect_tx(bar, __popc(on) * box * D);  // the slot's one arrival
                        if (++slot == C::NRAW) slot = 0, par ^= 1;
                    }
                }
                if (!ok || !advance<T>(a, p)) break;
            }
            if (!ok) {  // gave up: leave what TMA copies are in flight (microseconds) a millisecond
                for (int i = 0; i < 100; ++i) __nanosleep(10000);
            }
        } else if (F8 && warp == 15) {
            // ------------------------------------------------------------ 8 bits: the keys' scales, for the softmax
            constexpr int NK = BN / 32;  // keys per lane
            uint32_t tile = 0;
            bool ok = true;
            for (;;) {
                const int t0 = p.t0, t1 = p.t1, i0 = p.qt * a.tq, ntok = min(a.tq, p.s.m - i0);
                const int kend = min(t1 * BN, p.s.L - p.s.m + i0 + ntok);
                long long next[NK];
                auto entries = [&](int t) {
    #pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        const int pos = t * BN + i * 32 + lane;
                        next[i] = t < t1 && pos < kend ? page_entry(a, p.n, pos) : 0;
                    }
                };
                float ks[NK], vs[NK];  // 1 past the keys, where no weight is
                auto load = [&](int t) {
    #pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        const int pos = t * BN + i * 32 + lane;
                        const long long off = t < t1 && pos < kend ? row_of(a, next[i], p.h, pos) : -1;
                        ks[i] = off < 0 ? 1.f : a.ks[off];
                        vs[i] = off < 0 ? 1.f : a.vs[off];
                    }
                };
                entries(t0);
                load(t0);
                entries(t0 + 1);
                for (int t = t0; t < t1 && ok; ++t, ++tile) {
                    float k[NK], lv[NK], iv[NK];
    #pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        k[i] = ks[i];
                        lv[i] = fast_log2(vs[i]);
                        iv[i] = fast_rcp(vs[i]) * kUnlift;
                    }
                    load(t + 1);
                    entries(t + 2);
                    ok = warp_wait(SC_EMPTY + tile % C::SCN, (tile / C::SCN & 1) ^ 1);
                    if (!ok) break;
                    float* sc = reinterpret_cast<float*>(sm + C::OFF_SC) + tile % C::SCN * (3 * BN);
    #pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        sc[i * 32 + lane] = k[i];
                        sc[BN + i * 32 + lane] = lv[i];
                        sc[2 * BN + i * 32 + lane] = iv[i];
                    }
                    warp_arrive(SC_FULL + tile % C::SCN);
                }
                if (!ok || !advance<T>(a, p)) break;
            }
        } else if (warp == 12 && elect()) {
            // ------------------------------------------------------------ MMA issue
            // One elected lane (elect.sync, which the compiler knows to leave one: an MMA takes its descriptors from uniform
            // registers, and behind a branch on the lane index each one's operands are moved there first, which made
            // the issue twice as long as the products).
            constexpr uint32_t FMT = MF16 ? 0u : (1u << 7) | (1u << 10);
            constexpr uint32_t ID_S = (tc::idesc_bf16(128, BN, 0, 0, 0) & ~((1u << 7) | (1u << 10))) | FMT;
            constexpr uint32_t ID_O = (tc::idesc_bf16(128, D, 0, 1, 0) & ~((1u << 7) | (1u << 10))) | FMT;
            const uint32_t tmu = tm;
            const uint64_t dq = (tc::sdesc(sb, 16, 1024)), dk = (tc::sdesc(sb + C::OFF_KV, 16, 1024));
            const uint64_t dv = (tc::sdesc(sb + C::OFF_KV, BN * 128, 1024));
            uint32_t unit = 0, np[2] = {0, 0}, nr[2] = {0, 0};
            uint32_t ks = 0, kp = 0, vs = 1, vp = 0;  // stage and parity of the next K tile, of the next V tile
            uint32_t sc_in = 0, sc_out = 0;           // 8 bits: tiles whose scales have come, have been used
            auto step = [](uint32_t& stage, uint32_t& parity) {
                stage += 2;
                if (stage >= NST) {
                    stage -= NST;
                    parity ^= 1;
                }
            };
            bool ok = true;
            for (;;) {
                const int t0 = p.t0, t1 = p.t1;
                const int rows = min(a.tq, p.s.m - p.qt * a.tq) * a.G;
                const bool full = (SLOTS == 2 && rows > 128 ? 1u : 0u) != 0;
                const int nops = static_cast<int>((static_cast<uint32_t>(full ? 2 * (t1 - t0) : t1 - t0)));
                auto issue_s = [&](int s) {
                    const int b = s & 1;
                    if ((!full || !b) && !one_wait(KV_FULL + ks, kp)) return false;  // its tile's first product
                    const uint64_t qa = dq + (full && b ? C::QTILE >> 4 : 0u), ka = dk + ks * (C::TILE >> 4);
                    const bool last = !full || b;  // of this K tile's products
                    {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            if constexpr (C::QTM) tc::mma_bf16_ts(tmu + C::TM_S + b * C::TM_SB, tmu + C::TM_Q + 8 * k, ka + ((k >> 2) * (BN * 128) + (k & 3) * 32) / 16, ID_S, k > 0);
                            else tc::mma_bf16(tmu + C::TM_S + b * C::TM_SB, qa + ((k >> 2) * 16384 + (k & 3) * 32) / 16,
                                         ka + ((k >> 2) * (BN * 128) + (k & 3) * 32) / 16, ID_S, k > 0);
                        // S stands for the tile's scales too, and P for their having been read: even a wait that is over
                        // takes some 200 clocks, which this lane has and the softmax has not (windows: 117 -> 115 us)
                        if (F8 && (!full || !b)) {
                            if (!one_wait(SC_FULL + sc_in % C::SCN, sc_in / C::SCN & 1)) return false;
                            ++sc_in;
                        }
                        tc::commit(&bars[TB_S0 + b]);
                        if (last) tc::commit(&bars[KV_EMPTY + ks]);
                        if (!C::QTM && s == nops - 1) tc::commit(&bars[TB_QE]);
                    }
                    if (last) step(ks, kp);
                    return true;
                };
                ok = one_wait(TB_QF, unit & 1);
                ok = ok && issue_s(0) && (nops < 2 || issue_s(1));
                for (int s = 0; s < nops && ok; ++s) {
                    const int b = s & 1, o = SLOTS == 2 ? b : 0;
                    if (C::PSEP && s + 2 < nops) {  // S(s) has been read
                        ok = one_wait(TB_R0 + b, nr[b] & 1) && issue_s(s + 2);
                        if (!ok) break;
                    }
                    ++nr[b];
                    const bool fresh = SLOTS == 2 ? s < 2 : s == 0, last = !full || b;
                    ok = ((full && b) || one_wait(KV_FULL + vs, vp)) && (!fresh || one_wait(TB_OF0 + o, (unit & 1) ^ 1)) &&
                         one_wait((C::HALF ? TB_H0 : TB_P0) + b, np[b] & 1);
                    if (!ok) break;
                    ++np[b];
                    const uint64_t va = dv + vs * (C::TILE >> 4);
                    {
#pragma unroll
                        for (int k = 0; k < BN / 16; ++k) {
                            // the first half of P came first; now the rest
                            if (C::HALF && k == BN / 32 && !(ok = one_wait(TB_P0 + b, np[b] - 1 & 1))) break;
                            tc::mma_bf16_ts(tmu + C::TM_O + o * D, tmu + C::TM_P + b * C::TM_PB + 8 * k, va + k * (2048 / 16), ID_O,
                                            !fresh || k > 0);
                        }
                        if (!ok) break;
                        if (F8 && last) {
                            tc::mbar_arrive(&bars[SC_EMPTY + sc_out % C::SCN]);
                            ++sc_out;
                        }
                        tc::commit(&bars[TB_OD0 + b]);
                        if (last) tc::commit(&bars[KV_EMPTY + vs]);
                    }
                    if (last) step(vs, vp);
                    if (!C::PSEP && s + 2 < nops) ok = issue_s(s + 2);
                }
                if (!ok) break;
                ++unit;
                if (!advance<T>(a, p)) break;
            }
            // nothing of this CTA's may be in flight when it ends, its barriers' arrivals included
            {
                tc::commit(&bars[TB_DRAIN]);
                tc::mbar_wait(&bars[TB_DRAIN], 0, kWaitPolls);
            }
        }
    } else if (wg < SLOTS) {
        // ------------------------------------------------------------ softmax: one row per thread
        regs_up<kRegsSoftmax>();
        const int row = tid & 127;
        const uint32_t trow = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t unit = 0, ns[2] = {0, 0}, odp = 0, nml = 0, tiles = 0;
        (void)tiles;
        for (;;) {
            const int t0 = p.t0, t1 = p.t1;
            const int i0 = p.qt * a.tq, rows = min(a.tq, p.s.m - i0) * a.G;
            const bool full = SLOTS == 2 && rows > 128;
            const int nops = full ? 2 * (t1 - t0) : t1 - t0;
            const int r = (full ? wg * 128 : 0) + row;
            const bool live = r < rows, some = __any_sync(kFullMask, live);
            const int vis = live ? p.s.L - p.s.m + i0 + r / a.G + 1 : 0;  // keys that this row sees
            float c = a.scale_log2;
            if constexpr (C::QTM) {
                // this row's query into TMEM (the last unit's products with it are done: S of all of them was read)
                if (some) {
                    const uint4* src = reinterpret_cast<const uint4*>(a.q + (p.s.q0 + i0 + (live ? r / a.G : 0)) * a.q_stride +
                                                                      static_cast<long long>(p.h * a.G + (live ? r % a.G : 0)) * D);
                    float up = 1.f;
                    if constexpr (F8) {
                        float mx = 0.f;
#pragma unroll 8
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 q4 = live ? src[i] : make_uint4(0, 0, 0, 0);
                            const uint32_t x[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = unpack2<F16>(x[j]);
                                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                            }
                        }
                        up = row_up(mx);
                        c *= 1.f / up;
                    }
#pragma unroll 2
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint4 q4 = live ? src[4 * i + k] : make_uint4(0, 0, 0, 0);
                            w[4 * k] = q4.x;
                            w[4 * k + 1] = q4.y;
                            w[4 * k + 2] = q4.z;
                            w[4 * k + 3] = q4.w;
                        }
                        if constexpr (F8) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float2 f = unpack2<F16>(w[k]);
                                w[k] = pack2<true>(f.x * up, f.y * up);
                            }
                        }
                        __syncwarp();
                        tm_st16(trow + C::TM_Q + i * 16, w);
                    }
                    tc::wait_st();
                }
                tc::fence_before();
                warp_arrive(TB_QF);
            } else if constexpr (F8) {
                if (!warp_wait(TB_QF, unit & 1)) break;
                c = reinterpret_cast<const float*>(sm + C::OFF_RS)[(unit & 1) * C::R + r];
                // The next queries wait for this: a unit of one or two operations has all its products with Q done without
                // the softmax, which could still be in the unit before, and its wait above meet the phase after the one it
                // means (the same parity as the phase before).
                warp_arrive(TB_QE);
            }
            float ref = -INFINITY, l = 0.f;
            bool ok = true;
            int done = 0;  // this slot's operations of the unit
            // Operation s's product with V is done.  Each buffer has a barrier, of which one phase at most is pending: S(s)
            // was read, and the product before on this buffer came before it.  (A barrier for both could be two phases
            // on, or none, which a wait for a parity takes for the same.)
            auto product = [&](int s) { return warp_wait(TB_OD0 + (s & 1), (odp >> (s & 1) ^ s >> 1) & 1); };
            for (int s = SLOTS == 2 ? wg : 0; s < nops; s += SLOTS, ++done) {
                const int b = s & 1, tile = full ? s >> 1 : s, o = SLOTS == 2 ? b : 0;
                const uint32_t ts = trow + C::TM_S + b * C::TM_SB;
                const float* sc = nullptr;
                if constexpr (F8) {
                    sc = reinterpret_cast<const float*>(sm + C::OFF_SC) + (tiles + tile) % C::SCN * (3 * BN);
                }
                ok = warp_wait(TB_S0 + b, ns[b] & 1);
                if (!ok) break;
                ++ns[b];
                if (some) {
                    const int lim = vis - (t0 + tile) * BN;  // visible keys of the tile
                    const bool mask = __any_sync(kFullMask, lim < BN);
                    float y[BN];
#pragma unroll
                    for (int ch = 0; ch < BN / 32; ++ch) tm_ld32(ts + ch * 32, y + ch * 32);
                    tc::wait_ld();
                    if constexpr (C::PSEP) {
                        tc::fence_before();
                        warp_arrive(TB_R0 + b);
                    }
                    // y_j = raw_j times `times`, which is not negative
                    float times = fabsf(c);
                    if constexpr (F8) {
                        times = 1.f;
#pragma unroll
                        for (int i = 0; i < BN; i += 4) {
                            const float4 ks = *reinterpret_cast<const float4*>(sc + i);
                            const float4 lv = *reinterpret_cast<const float4*>(sc + BN + i);
                            pair_fma(y + i, y + i, c, ks.x, ks.y, lv.x, lv.y);
                            pair_fma(y + i + 2, y + i + 2, c, ks.z, ks.w, lv.z, lv.w);
                        }
                        if (mask) {
#pragma unroll
                            for (int i = 0; i < BN; ++i)
                                if (i >= lim) y[i] = -INFINITY;
                        }
                    } else if (mask) {
                        times = 1.f;
#pragma unroll
                        for (int i = 0; i < BN; ++i) y[i] = i >= lim ? -INFINITY : y[i] * c;
                    } else if (c < 0.f) {
#pragma unroll
                        for (int i = 0; i < BN; ++i) y[i] = -y[i];
                    }
                    float m4[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
                    for (int i = 4; i < BN; i += 8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) m4[j] = i + 4 + j < BN ? fmaxf(fmaxf(m4[j], y[i + j]), y[i + 4 + j]) : fmaxf(m4[j], y[i + j]);
                    }
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * times;
                    if (C::PSEP && done > 0) {  // P's columns are free
                        ok = product(s - SLOTS);
                        if (!ok) break;
                    }
                    if (__any_sync(kFullMask, mx > ref + kRefSlack)) {
                        const float to = fmaxf(ref, mx);
                        const float f = to == -INFINITY ? 1.f : fast_exp2(ref - to);
                        ref = to;
                        l *= f;
                        if (done > 0) {  // what has been accumulated so far
                            ok = C::PSEP || product(s - SLOTS);
                            if (!ok) break;
#pragma unroll 1
                            for (int ch = 0; ch < D / 16; ++ch) {
                                float v[16];
                                tc::ld16(trow + C::TM_O + o * D + ch * 16, v);
                                tc::wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] *= f;
                                tc::st16(trow + C::TM_O + o * D + ch * 16, v);
                            }
                        }
                    }
                    const float use = ref == -INFINITY ? 0.f : ref - kLift;
                    float l2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ch = 0; ch < BN / 32; ++ch) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float* x = y + ch * 32 + i;
                            pair_exp2(x, times, -use);
                            pair_exp2(x + 2, times, -use);
                            if constexpr (F8) {
                                const float4 iv = *reinterpret_cast<const float4*>(sc + 2 * BN + ch * 32 + i);
                                pair_mac(l2, x, iv.x, iv.y);
                                pair_mac(l2 + 2, x + 2, iv.z, iv.w);
                            } else {
                                pair_add(l2, x);
                                pair_add(l2 + 2, x + 2);
                            }
                            w[i / 2] = pack2<MF16>(x[0], x[1]);
                            w[i / 2 + 1] = pack2<MF16>(x[2], x[3]);
                        }
                        tm_st16(trow + C::TM_P + b * C::TM_PB + ch * 16, w);
                        if (C::HALF && ch == BN / 64 - 1) {  // half of P: its products can start
                            tc::wait_st();
                            tc::fence_before();
                            warp_arrive(TB_H0 + b);
                        }
                    }
                    l += (l2[0] + l2[1]) + (l2[2] + l2[3]);
                    tc::wait_st();
                } else if (SLOTS == 2) {
                    if (C::PSEP) {
                        warp_arrive(TB_R0 + b);
                        // the barrier's phases are waited for one by one
                        ok = done == 0 || product(s - SLOTS);
                        if (!ok) break;
                    }
                    if (C::HALF) warp_arrive(TB_H0 + b);
                }
                tc::fence_before();
                warp_arrive(TB_P0 + b);
            }
            if (!ok) break;
            tiles += t1 - t0;

            // ---- the unit's rows
            if constexpr (!F8) l *= kUnlift;
            const bool both = SLOTS == 2 && !full;  // the slots hold two parts of the same rows
            float f0 = 1.f, f1 = 0.f;
            if (both && wg == 1) {
                ok = warp_wait(TB_ME, (nml & 1) ^ 1);
                if (!ok) break;
                ml_s[row][0] = ref;
                ml_s[row][1] = l;
                warp_arrive(TB_MF);
            } else {
                if (both) {
                    ok = warp_wait(TB_MF, nml & 1);
                    if (!ok) break;
                    const float ref1 = ml_s[row][0], l1 = ml_s[row][1];
                    warp_arrive(TB_ME);
                    const float top = fmaxf(ref, ref1);
                    if (top != -INFINITY) {
                        f0 = fast_exp2(ref - top);
                        f1 = fast_exp2(ref1 - top);
                    }
                    l = l * f0 + l1 * f1;
                    ref = top;
                }
                const int o = SLOTS == 2 ? wg : 0;
                // this accumulator's last product (one accumulator: the unit's last), and the other slot's
                auto newest = [&](int b) { return nops - 1 - ((nops - 1 ^ b) & 1); };  // the last operation in buffer b
                ok = product(SLOTS == 2 ? newest(wg) : nops - 1) && (!both || nops < 2 || product(newest(1)));
                if (!ok) break;
                if (some) {
                    const bool whole = t0 == 0 && t1 == p.nk;
                    const float inv = l > 0.f || l != l ? kUnlift / l : 0.f;
                    const long long orow = (p.s.q0 + i0 + r / a.G) * a.Hq + p.h * a.G + r % a.G;
                    float* part = a.part + (static_cast<long long>(blockIdx.x) * 2 + (t0 > 0 ? 0 : 1)) *
                                               (static_cast<long long>(C::R) * (D + 2));
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        float v[32];
                        tm_ld32(trow + C::TM_O + o * D + ch * 32, v);
                        tc::wait_ld();
                        if (both && nops > 1) {
                            float u[32];
                            tm_ld32(trow + C::TM_O + D + ch * 32, u);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = fmaf(f1, u[i], f0 * v[i]);
                        }
                        if (live && whole) {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + ch * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                dst[i] = make_uint4(pack2<F16>(v[8 * i] * inv, v[8 * i + 1] * inv), pack2<F16>(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                                    pack2<F16>(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack2<F16>(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
                        } else if (live) {
                            float4* dst = reinterpret_cast<float4*>(part + static_cast<long long>(r) * D + ch * 32);
#pragma unroll
                            for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                        __syncwarp();
                    }
                    if (live) {
                        if (!whole) {
                            part[static_cast<long long>(C::R) * D + r] = ref;
                            part[static_cast<long long>(C::R) * (D + 1) + r] = l;
                        } else if (a.lse) {
                            a.lse[orow] = l == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(l)) * kLn2;
                        }
                    }
                }
                tc::fence_before();
                warp_arrive(TB_OF0 + o);
                if (both) warp_arrive(TB_OF0 + 1);
            }
            if (both) ++nml;
            odp ^= ((nops + 1) / 2 & 1) | (nops / 2 & 1) << 1;  // parities of the buffers' operations so far
            ++unit;
            if (!advance<T>(a, p)) break;
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 12) tc::tmem_dealloc(tm, 512);
    if (tid == 0 && most_polls == 0) atomicOr(a.status, kStatusTimeout);
}

}  // namespace attn
}  // namespace gdn
