// attn_rows.cuh -- attn_paged for few query rows per key head (single tokens): tiles of 16 rows.
//
// Bound: the cache is read once from HBM and each key row meets at most 16 query rows, about 16
// operations per byte, so the time is the bytes' time.  What the kernel has to do is keep enough of
// them in flight and stay out of their way.  Hence: four independent warps per CTA, each with its own
// ring of stages of TK = 16 or 32 keys (no block barrier inside a unit); warp w takes keys TK w .. TK w + TK - 1
// of each tile of 4 TK keys and keeps its own reference, sum and accumulator, joined once per unit through
// shared memory.  The products run on mma.sync m16n8k16: its 16 rows are the whole tile, whereas a
// tcgen05.mma would compute 128 rows for them and add a TMEM round trip per tile.
//
// 8-bit caches (F8): e4m3 values widen exactly to binary16, so both products run on binary16 operands.
// A query row is first multiplied by a power of two that brings its largest element to 2^13 .. 2^14
// (bf16 elements down to 2^-27 of the row's largest stay exact); the power, the key's scale and the
// softmax scale multiply the fp32 product.  The value's scale moves into the exponent,
//     p'_j = 2^{y_j + log2(vs_j) - ref + kLift},   l = 2^-kLift sum p'_j / vs_j,   acc = sum p'_j v_j,
// so that p' fits binary16 whatever the scales' sizes are.
//
// Measured, one token each of 64 sequences: 16 bits, up to 8192 keys of 8 x 128, 187 us, 97 % of a copy's rate; 8
// bits, up to 16384 keys of 4 x 128, 112 us, 84 %: there the widening's and the products' instructions take as long.
#pragma once

#include "attn.cuh"
#include "attn_mma.cuh"
#include "tcgen05.cuh"

namespace gdn {
namespace attn {

constexpr int kRowsTile = 16;   // rows per query tile
constexpr int kRowsNT = 128;

template <int D, bool F8>
struct RowsCfg {
    static constexpr int ROWB = F8 ? D : 2 * D;      // bytes per cached row
    static constexpr int CH = ROWB / 16;             // 16-byte chunks per cached row
    static constexpr int LINE = ROWB < 128 ? ROWB : 128;  // bytes of a row that stand together
    static constexpr int COLS = ROWB / LINE;         // a stage's rows as COLS blocks of TK lines
    // keys per step and warp.  8 bits: a step of 16 took 560 instructions, half of them not for its products
    static constexpr int TK = F8 && D <= 128 ? 32 : 16;
    static constexpr int BN = 4 * TK;                // keys per tile of the CTA
    static constexpr int STAGE = 2 * TK * ROWB;      // K rows, V rows
    // stages per warp: 64 to 100 KB per CTA, two or three CTAs per SM
    static constexpr int NS = D == 256 ? 3 : (D == 128 ? (F8 ? 2 : 3) : (F8 ? 3 : 4));
    static constexpr int RING = NS * STAGE * 4;
    static constexpr int SCALE = 8 * TK;             // a stage's scales: K, V
    static constexpr int SCALES = F8 ? NS * 4 * SCALE : 0;
    static constexpr int MERGE = 4 * 16 * D * 4;
    static constexpr int SMEM = (RING + SCALES > MERGE ? RING + SCALES : MERGE) + 1024;
    static constexpr int OCC = D == 256 ? (F8 ? 2 : 1) : (D == 128 ? (F8 ? 3 : 2) : 3);
};

// Byte offset of 16-byte chunk c of row r of a stage's rows: the layout that TMA writes with its 128-byte
// (64-byte) swizzle, in which eight rows at one chunk column, or eight consecutive chunks, fall on
// different banks.
template <class C>
__device__ __forceinline__ int rows_at(int r, int c) {
    if constexpr (C::LINE == 128) return (c >> 3) * (C::TK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, bool F16, bool F8>
__global__ void __launch_bounds__(kRowsNT, RowsCfg<D, F8>::OCC) attn_rows_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using C = RowsCfg<D, F8>;
    constexpr bool MF16 = F16 || F8;  // operand type of the products
    constexpr int TK = C::TK, BN = C::BN, NS = C::NS, CH = C::CH, KS = D / 16, NT = TK / 8;
    typedef Tiling<BN, 1, kRowsTile> RowsTiling;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanSmem plan_s;
    __shared__ float m_s[4][16], l_s[4][16];
    __shared__ uint64_t full[4][NS];  // a stage filled by TMA
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;  // fragment row and column group

    Walk p;
    long long per;
    const bool busy = plan<RowsTiling, kRowsNT>(a, plan_s, p, per);
    pdl_launch();
    if (!busy) {
        if (tid == 0) leave_no_join(a);
        return;
    }

    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t ring_a = smem_addr(smem) + warp * (NS * C::STAGE);
    const uint32_t scale_a = smem_addr(smem) + C::RING + warp * (NS * C::SCALE);
    float* merge = reinterpret_cast<float*>(smem);
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) tc::mbar_init(&full[warp][i], 1);
        tc::fence_proxy_async();
    }
    __syncwarp();
    uint32_t phase = 0;     // of the stages' barriers
    bool gave_up = false;

    for (;;) {
        const int t0 = p.t0, t1 = p.t1;
        const int i0 = p.qt * a.tq;
        const int ntok = min(a.tq, p.s.m - i0), rows = ntok * a.G;
        const int vis0 = p.s.L - p.s.m + i0 + 1;      // keys that token i0 sees
        const int kend = min(t1 * BN, vis0 + ntok - 1);  // one past the last key of this segment

        // ---- query fragments: rows g and g + 8 ----
        uint32_t qf[KS][4];
        float rscale[2];
        int vis[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = g + 8 * half;
            const bool live = r < rows;
            const int tok = live ? r / a.G : 0;
            vis[half] = live ? vis0 + tok : 0;
            const uint16_t* src = a.q + (p.s.q0 + i0 + tok) * a.q_stride + static_cast<long long>(p.h * a.G + (live ? r - tok * a.G : 0)) * D;
            rscale[half] = a.scale_log2;
            if constexpr (!F8) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t* s32 = reinterpret_cast<const uint32_t*>(src + k * 16 + t * 2);
                    qf[k][half] = live ? s32[0] : 0u;
                    qf[k][half + 2] = live ? s32[4] : 0u;
                }
            } else {
                // K step 4 kk + j holds, in thread column group t, features kk 64 + t 16 + 4 j + 0 .. 3
                float mx = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 64; ++kk) {
                    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (live) {
                        w[0] = *reinterpret_cast<const uint4*>(src + kk * 64 + t * 16);
                        w[1] = *reinterpret_cast<const uint4*>(src + kk * 64 + t * 16 + 8);
                    }
                    const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        qf[4 * kk + j][half] = x[2 * j];
                        qf[4 * kk + j][half + 2] = x[2 * j + 1];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = unpack2<F16>(x[2 * j + i]);
                            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
                const float up = row_up(mx);
                rscale[half] *= 1.f / up;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = unpack2<F16>(qf[k][half + 2 * i]);
                        qf[k][half + 2 * i] = pack2<true>(f.x * up, f.y * up);
                    }
                }
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // `ref` is the reference less kLift until the unit's end, which saves a subtraction per step
        float ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};

        // ---- this warp's steps: keys (t0 + s) BN + warp TK .. + TK - 1, while any is below kend ----
        const int first = t0 * BN + warp * TK;
        const int steps = kend > first && !gave_up ? (kend - first + BN - 1) / BN : 0;
        // 8 bits, pages that 16 divides: TMA, by boxes of a.box rows, of which one page holds each; lane i looks
        // up and copies box i.  Else (any page size) cp.async: every lane looks up a row, and rows past kend are
        // zero-filled.  16-bit rows take that way always: it keeps as many bytes in flight, and is ready earlier
        // (64 sequences of up to 8192 keys, 8 x 128: 184 us, by TMA 188).
        const bool tma = F8 && a.box >= 16;
        const int mine = tma ? lane * a.box : lane & (TK - 1);  // the row, or the first of a box, of this lane
        auto entry = [&](int s) -> long long {
            const int pos = first + s * BN + mine;
            return s < steps && mine < TK && pos < kend ? page_entry(a, p.n, pos) : 0;
        };
        long long next = entry(0);
        auto issue = [&](int s) {
            if (s < steps) {
                const int pos = first + s * BN + mine;
                const long long off = mine < TK && pos < kend ? row_of(a, next, p.h, pos) : -1;
                next = entry(s + 1);
                const int st = s % NS;
                const uint32_t dst = ring_a + st * C::STAGE, sdst = scale_a + st * C::SCALE;
                if (tma) {
                    uint64_t* bar = &full[warp][st];
                    const unsigned on = __ballot_sync(kFullMask, off >= 0);
                    if (lane == 0) tc::mbar_expect_tx(bar, __popc(on) * a.box * (2 * C::ROWB + 8));
                    __syncwarp();
                    if (off >= 0) {
                        const int r = lane * a.box;
#pragma unroll
                        for (int x = 0; x < C::COLS; ++x) {
                            tma_load_2d(dst + x * (TK * 128) + r * C::LINE, &maps.k, x * C::LINE, static_cast<int>(off), bar);
                            tma_load_2d(dst + TK * C::ROWB + x * (TK * 128) + r * C::LINE, &maps.v, x * C::LINE, static_cast<int>(off), bar);
                        }
                        tc::bulk_load(sdst + r * 4, a.ks + off, a.box * 4, bar);
                        tc::bulk_load(sdst + TK * 4 + r * 4, a.vs + off, a.box * 4, bar);
                    }
                } else {
                    if constexpr (F8) {
                        if (lane < TK) {
                            cp_async4(sdst + lane * 4, a.ks + (off < 0 ? 0 : off), off >= 0);
                            cp_async4(sdst + TK * 4 + lane * 4, a.vs + (off < 0 ? 0 : off), off >= 0);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < CH * TK / 32; ++i) {
                        const int idx = i * 32 + lane, r = idx / CH, c = idx % CH;
                        const long long ro = __shfl_sync(kFullMask, off, r);
                        const long long byte = (ro < 0 ? 0 : ro * C::ROWB) + c * 16;
                        const uint32_t d = dst + rows_at<C>(r, c);
                        cp_async16(d, static_cast<const uint8_t*>(a.kc) + byte, ro >= 0);
                        cp_async16(d + TK * C::ROWB, static_cast<const uint8_t*>(a.vc) + byte, ro >= 0);
                    }
                }
            }
            if (!tma) cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) issue(s);

        for (int s = 0; s < steps; ++s) {
            const int st = s % NS, base = first + s * BN;
            const uint32_t kst = ring_a + st * C::STAGE, vst = kst + TK * C::ROWB, sst = scale_a + st * C::SCALE;
            if (tma) {
                if (!tc::mbar_wait(&full[warp][st], phase >> st & 1, a.polls)) {
                    atomicOr(a.status, kStatusTimeout);
                    gave_up = true;
                }
                phase ^= 1u << st;
                if (base + TK > kend) {  // what the page holds past the keys must not meet a weight of zero
                    __syncwarp();
                    for (int i = lane; i < TK * CH; i += 32)
                        if (base + i / CH >= kend) sts128(vst + rows_at<C>(i / CH, i % CH), make_uint4(0, 0, 0, 0));
                    tc::fence_proxy_async();  // before TMA writes here again
                }
            } else {
                cp_async_wait<NS - 2>();
            }
            if (__any_sync(kFullMask, gave_up)) {
                gave_up = true;
                // this step's copies and the next ones' are in flight: they land before the warp goes on
                for (int k = s; k < min(s + NS - 1, steps); ++k)
                    tc::mbar_wait(&full[warp][k % NS], (phase >> k % NS & 1) ^ (k == s), kWaitPolls);
                break;
            }
            __syncwarp();  // all lanes' copies and zeros are in place, and the previous step has read its stage
            issue(s + NS - 1);  // into the stage that the previous step has read

            float sc[NT][4] = {};
            if constexpr (!F8) {
                const int mi = lane >> 3, tok = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b[4];
                    ldsm4(b, kst + rows_at<C>(tok, 2 * k + (mi & 1)));
                    mma16816<MF16>(sc[0], qf[k], b[0], b[1]);
                    mma16816<MF16>(sc[1], qf[k], b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 64; ++kk) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 w = lds128(kst + rows_at<C>(nt * 8 + g, kk * 4 + t));
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma16816<true>(sc[nt], qf[4 * kk + j], e4m3_lo(x[j]), e4m3_hi(x[j]));
                    }
                }
            }

            // ---- y = s log2(e), masked; 8-bit values: plus log2 of the value's scale ----
            float iv[NT][2];
            if constexpr (F8) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 ks = lds64(sst + (nt * 8 + 2 * t) * 4), vs = lds64(sst + TK * 4 + (nt * 8 + 2 * t) * 4);
                    const float lv[2] = {fast_log2(vs.x), fast_log2(vs.y)};
                    iv[nt][0] = fast_rcp(vs.x) * kUnlift;
                    iv[nt][1] = fast_rcp(vs.y) * kUnlift;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // the scales first: either may be as large or as small as numbers get
                        sc[nt][2 * half] = fmaf(sc[nt][2 * half], rscale[half] * ks.x, lv[0]);
                        sc[nt][2 * half + 1] = fmaf(sc[nt][2 * half + 1], rscale[half] * ks.y, lv[1]);
                    }
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[nt][i] *= a.scale_log2;
            }
            if (base + TK > vis0 || base + TK > kend) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int pos = base + nt * 8 + 2 * t + (i & 1);
                        if (pos >= vis[i >> 1] || pos >= kend) sc[nt][i] = -INFINITY;
                        if (F8 && pos >= kend) iv[nt][i & 1] = 0.f;  // no key, no scale
                    }
            }
            float mx[2], use[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x = fmaxf(sc[0][2 * half], sc[0][2 * half + 1]);
#pragma unroll
                for (int nt = 1; nt < NT; ++nt) x = fmaxf(x, fmaxf(sc[nt][2 * half], sc[nt][2 * half + 1]));
                x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 1));
                mx[half] = fmaxf(x, __shfl_xor_sync(kFullMask, x, 2));
            }
            // rows move their reference when a score is kRefSlack above it (the first time: above -inf)
            const bool up = mx[0] > ref[0] + (kLift + kRefSlack) || mx[1] > ref[1] + (kLift + kRefSlack);
            if (__any_sync(kFullMask, up)) {
                float f[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float to = fmaxf(ref[half], mx[half] - kLift);
                    f[half] = to == -INFINITY ? 1.f : fast_exp2(ref[half] - to);
                    ref[half] = to;
                    lsum[half] *= f[half];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= f[0];
                    o[i][1] *= f[0];
                    o[i][2] *= f[1];
                    o[i][3] *= f[1];
                }
            }
            use[0] = ref[0] == -INFINITY ? 0.f : ref[0];
            use[1] = ref[1] == -INFINITY ? 0.f : ref[1];
            uint32_t pf[NT / 2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float x = fast_exp2(sc[nt][2 * half] - use[half]), y = fast_exp2(sc[nt][2 * half + 1] - use[half]);
                    if constexpr (F8) lsum[half] = fmaf(x, iv[nt][0], fmaf(y, iv[nt][1], lsum[half]));
                    else lsum[half] += x + y;
                    pf[nt / 2][2 * (nt & 1) + half] = pack2<MF16>(x, y);
                }
            }

            const int mi = lane >> 3;
#pragma unroll
            for (int kg = 0; kg < TK / 16; ++kg) {
                const int vtok = kg * 16 + (mi & 1) * 8 + (lane & 7);
                if constexpr (!F8) {
#pragma unroll
                    for (int dc = 0; dc < D / 16; ++dc) {
                        uint32_t b[4];
                        ldsm4t(b, vst + rows_at<C>(vtok, 2 * dc + (mi >> 1)));
                        mma16816<MF16>(o[2 * dc], pf[kg], b[0], b[1]);
                        mma16816<MF16>(o[2 * dc + 1], pf[kg], b[2], b[3]);
                    }
                } else {
                    // a chunk's even features make one 8-column tile, its odd features another
#pragma unroll
                    for (int c2 = 0; c2 < D / 32; ++c2) {
                        uint32_t b[4];
                        ldsm4t(b, vst + rows_at<C>(vtok, 2 * c2 + (mi >> 1)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo = __byte_perm(b[2 * i], 0, 0x3120), hi = __byte_perm(b[2 * i + 1], 0, 0x3120);
                            mma16816<true>(o[4 * c2 + 2 * i], pf[kg], e4m3_lo(lo), e4m3_lo(hi));
                            mma16816<true>(o[4 * c2 + 2 * i + 1], pf[kg], e4m3_hi(lo), e4m3_hi(hi));
                        }
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            lsum[half] += __shfl_xor_sync(kFullMask, lsum[half], 1);
            lsum[half] += __shfl_xor_sync(kFullMask, lsum[half], 2);
            if constexpr (!F8) lsum[half] *= kUnlift;
            ref[half] += kLift;
        }

        // ---- join the four warps: accumulators through shared memory (the rings are drained) ----
        __syncthreads();
        if (t == 0) {
            m_s[warp][g] = ref[0];
            m_s[warp][g + 8] = ref[1];
            l_s[warp][g] = lsum[0];
            l_s[warp][g + 8] = lsum[1];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float* dst = merge + (warp * 16 + g + 8 * half) * D;
            if constexpr (!F8) {
#pragma unroll
                for (int nt = 0; nt < D / 8; ++nt)
                    *reinterpret_cast<float2*>(dst + ((nt * 8 + 2 * t) ^ (g << 2 & 24))) = make_float2(o[nt][2 * half], o[nt][2 * half + 1]);
            } else {
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    *reinterpret_cast<float4*>(dst + ((c * 16 + 4 * t) ^ (g << 2 & 24))) =
                        make_float4(o[2 * c][2 * half], o[2 * c + 1][2 * half], o[2 * c][2 * half + 1],
                                    o[2 * c + 1][2 * half + 1]);
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == p.nk;
        float* part = a.part + (static_cast<long long>(blockIdx.x) * 2 + (t0 > 0 ? 0 : 1)) * (16LL * (D + 2));
        constexpr int TPR = D / 4;  // threads per row, four columns each
        for (int r = tid / TPR; r < rows; r += kRowsNT / TPR) {
            const int col = (tid % TPR) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, m_s[w][r]);
            const float zero = top == -INFINITY ? 0.f : top;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = fast_exp2(m_s[w][r] - zero);
                const float4 v = *reinterpret_cast<const float4*>(merge + (w * 16 + r) * D + (col ^ ((r & 7) << 2 & 24)));
                l = fmaf(f, l_s[w][r], l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if (whole) {
                const float inv = l > 0.f || l != l ? kUnlift / l : 0.f;
                const long long row = (p.s.q0 + i0 + r / a.G) * a.Hq + p.h * a.G + r % a.G;
                uint2 w;
                w.x = pack2<F16>(acc.x * inv, acc.y * inv);
                w.y = pack2<F16>(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + col) = w;
                if (a.lse && col == 0) a.lse[row] = l == 0.f ? -INFINITY : (zero + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(part + r * D + col) = acc;
                if (col == 0) {
                    part[16 * D + r] = top;
                    part[16 * (D + 1) + r] = l;
                }
            }
        }
        if (tid == 0) leave_join(a, p, per);  // the last unit's stands
        if (!advance<RowsTiling>(a, p)) break;
        tc::fence_proxy_async();
        __syncthreads();  // the rings are written again
    }
}

}  // namespace attn
}  // namespace gdn
