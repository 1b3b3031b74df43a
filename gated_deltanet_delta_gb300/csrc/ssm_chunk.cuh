// ssm_chunk.cuh -- the state space scan over prompts, in chunks of 128 tokens on the tensor cores (tcgen05, accumulators in TMEM).
//
// With a_t = A dt_t and s <= t in a chunk whose first state is S:
//     y_t = sum_s (C_t . B_s) e^(a_(s+1) + .. + a_t) dt_s x_s + e^(a_1 + .. + a_t) C_t S^T + D x_t,
//     S' = e^(a_1 + .. + a_Q) S + sum_s e^(a_(s+1) + .. + a_Q) dt_s x_s (x) B_s.
// A CTA has 128 features of one segment of a sequence (two heads of 64 that share B and C, or one of 128) and walks its chunks:
//     G = C B^T (128 x 128 x N),  Y = C S^T (128 x 128 x N),  M X (128 x 64 x 128 per head of 64),
//     S = e^(..) S + X'^T B (128 x N x 128, three times),
// M = G with the weights of its pairs and X' = the rows of x with theirs, made by threads, which also join the output, e^(..) Y + M X + D x.
// S, G, M and Y fill TMEM (512 columns for N = 128; M X takes G's place); tiles of x, B and C come by TMA.
//
// A difference of running sums loses as many bits as the sums have, so they run over blocks of 32 tokens only, in which a pair's decay is the
// exponential of such a difference, and a step counts as at most 2^-128, which is zero here: a sum is at most 4096, its five levels of additions
// are off by less than 2^-12 together, and a weight by 2^-11 ln 2 (3.4e-4) where a block is full of such steps, a twelfth of what its
// rounding to bf16 may take.  A pair of tokens in two blocks has the product of two factors, the one of the row and
// its block, the other of the column, which also saves the exponentials: one per pair only inside the blocks.
//
// The state is an fp32 result and is carried for thousands of chunks, so X' is held in three bf16 parts, which leave nothing of fp32 out; M and
// the copy of S that Y is made from are rounded to bf16 (2^-8 of each product at most, like the output's own rounding).  With two parts a
// state is off by 2.5e-6 of its norm.  Over the pools of the two prompts below, against 64 bits: 3.2e-7 and 8e-8 (two parts: 1.0e-6 and
// 5.4e-7, in 333 and 227 us; token by token: 3.8e-7 and 3e-8).  Where one head has the tile to itself and B is half as wide, B takes the
// weights instead of x (B' below, also in three parts): half the threads' work, and room for all of the parts.
//
// Roles, 640 threads.  Sixteen workers' warps: a thread is a token (a TMEM lane) of M, of Y and of X', and a feature of the state.
// Warpgroups 0 and 1 (A) have M's diagonal blocks and the next ones and the high parts of X', 2 and 3 (B) the blocks further off, the
// others, and the state between two chunks; the output (D, the gate) is shared, 32 features each, and the decays' sums are made by
// the warps that have the least of M.  Warp 16 loads x, B and C, a lane of warp 17 issues what the outputs are made of and one of warp
// 18 the state's update, and warp 19 loads the gate and stores the output.  Per chunk c
//     A: M | X' high of c + 1 | output        B: M, X' middle and low | state of c + 1 | output.
// (B's output ahead of the state: 2 to 4 % less without a gate, 4 % more with one, whose rows come late in the place of the output.)
// Measured: four prompts of up to 8192 tokens, 64 heads of 64, N = 128, gated: 350 us, 5.5 us per chunk of the longest chain; one of
// 16384 tokens, 32 heads of 128, N = 64: 216 us.  No unit bounds it: a scheduler
// issues in 49 % of the cycles, the tensor core is at work in 24 %, the rest is the latency of four warps' instructions per scheduler and
// the hand-overs.  HBM would take 104 and 42 us, the tensor core 1.9 us a chunk.
//
// Segments.  A sequence is a chain, and a call with few sequences and heads has fewer chains than the GPU has SMs.  Long sequences are
// cut into segments that run side by side: a launch ahead (ssm_ahead_kernel) forms the states that all segments but the last end in
// from a zero state (the first from the pool's), and a segment starts from the sum of those ahead of it with their decays.  Those sums
// grow with the square of the segments, which ssm.cu keeps few: one prompt of 16384, 32768 and 131072 tokens, 64 heads of 64, N = 128, takes 271,
// 506 and 1901 us.
//
// Every wait is bounded (attn_tiles.cuh): one that runs out sets GDN_STATUS_TIMEOUT and the CTA's limit of polls to 0.  A CTA that gave
// up ends behind one more bounded wait for each product and copy that it has in flight, and leaves the pool's state as it is; one whose
// segment starts from what another did not come to write gives up too.
#pragma once

#include "attn_mma.cuh"
#include "ssm.cuh"
#include "tcgen05.cuh"
#include "tile_util.cuh"

namespace gdn {
namespace ssm {

constexpr int kChunk = 128;
constexpr int kChunkNT = 640;
constexpr int kSegment = 8;      // segments are multiples of so many chunks
constexpr int kWhole = 1 << 24;  // chunks per segment where no sequence is cut
// registers per thread: the launch's 96 x 5 warpgroups, parted as 104 x 4 for the workers and 64 for those that load and issue
constexpr int kRegsLaunch = 96, kRegsWork = 104, kRegsIssue = 64;
constexpr float kNoState = 1.f;        // in the place of a decay's logarithm, which is never positive: the state was not written
constexpr uint32_t kPolls = 1u << 22;  // the built-in limit of a wait (seconds)

template <int P, int S>
struct ChunkCfg {
    static constexpr uint32_t X = 32768, CB = kChunk * S * 2;  // bytes of a tile of x, of B or C
    // Whether B takes the weights of the state's products instead of x: where one head has the tile to itself and B is half as wide.
    static constexpr bool WB = P == 128 && S == 64;
    static constexpr int NB = S == 64 ? 2 : 1, NC = WB ? 2 : 1;  // buffers of B and of C; x has two
    static constexpr uint32_t OFF_H = 0, OFF_S = X;              // high parts; the state's copy
    // The middle parts come in the place of the state's copy and the low ones in C's, once those have been read; B's have places of their own.
    static constexpr uint32_t OFF_M = WB ? X + CB : X, OFF_L = WB ? CB : 2 * X;
    static constexpr uint32_t OFF_C = 2 * X, OFF_B = 3 * X, OFF_X = OFF_B + NB * CB, OFF_V = OFF_X + 2 * X;
    // per chunk (two in turn) and head: the decays' sums within blocks of 32 tokens, the columns' factors, dt (in the
    // exponent it would be lost beside a large sum), the blocks' sums
    static constexpr int VEC = 3 * kChunk + 16;
    // the gate's rows, and then the output's, of the last three blocks of 32: there is no room for the first
    static constexpr uint32_t OFF_Z = (OFF_V + 2 * 2 * VEC * 4 + 1023) / 1024 * 1024, ZBOX = 4096;
    static constexpr uint32_t USED = OFF_Z + 6 * ZBOX;
    static constexpr uint32_t SMEM = USED + 1024;
    static constexpr uint32_t TM_S = 0, TM_G = 128, TM_M = 256, TM_Y = 384;
};

// Barriers, two of each for the chunks in turn.
enum : int {
    CK_X = 0, CK_BC, CK_XE, CK_G, CK_CS, CK_UPH, CK_UPD, CK_MX0, CK_MX1, CK_V, CK_S, CK_XH, CK_XL, CK_M, CK_YF, CK_O, CK_Z, CK_ZE, CK_DRAIN, CK_N
};

struct Unit {
    long long begin;   // first token
    long long slot;    // of the state pool
    long long ws;      // first state of the sequence in the workspace
    int len, chunks;   // tokens, chunks
    int k;             // segment (piece) of its sequence
    int parts;         // segments of its sequence
    int found;
};

__device__ __forceinline__ void tma_store_2d(const void* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const void* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
// 8 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                 "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Eight floats at once, 32-byte aligned: a lane has a row of the state to itself, so that an instruction touches 32 lines whatever its width.
__device__ __forceinline__ void ld_state(const float* p, float* v) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_state(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
                 "f"(v[6]), "f"(v[7])
                 : "memory");
}
// A weight of a pair beyond bf16's range becomes its largest number: it may stand for an x of zero.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// WB: of a row of B times its weight, which may stand for an x of zero too.
template <bool WB>
__device__ __forceinline__ uint32_t pack_part(attn::f32x2 p) {
    float f[2];
    attn::unpair(p, f);
    return WB ? pack_weights(f[0], f[1]) : pack_bf16x2(f[0], f[1]);
}
// x, which the compiler does not know to be the same from chunk to chunk: what depends on it is computed where it is used, and does
// not take registers in between (they were spilled, and each reload from memory took some 300 clocks).
__device__ __forceinline__ int anew(int x) {
    asm volatile("" : "+r"(x));
    return x;
}
__device__ __forceinline__ float ex2(float x) { return attn::fast_exp2(x); }
// The logarithm (base 2) of a token's decay, for A to that base: not below -128, as ex2 is zero from there on (without the limit one step of
// thousands takes the digits of its block's other decays, and one that is no longer a number of fp32 makes them NaN); 0 for no token.  A NaN stays one.
__device__ __forceinline__ float log_decay(float A, float dt) {
    float a;
    asm("max.NaN.f32 %0, %1, 0fC3000000;" : "=f"(a) : "f"(A * dt));
    return dt > 0.f ? a : 0.f;
}

// The unit with number `rank`: one warp walks the sequences, twice: segments of a.seg chunks come first, then what is left of the
// sequences, so that the last to start are the short ones.  The walk has 32 sequences at a time and all of its SM wait: of 32 tokens each (64 heads
// of 64, N = 128) 256, 1024 and 4096 sequences take 0.84, 4.4 and 36 ms.  Ahead (AHEAD) are all segments but each sequence's last.  A sequence of
// more than a.seg chunks has states in the workspace: the pool's, then one for each segment ahead.
template <bool AHEAD>
__device__ __forceinline__ void find_unit(const SsmArgs& a, int rank, Unit& u) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    if (lane == 0) u.found = 0;
#pragma unroll 1
    for (int walk = AHEAD || a.seg < kWhole ? 0 : 1; walk < (AHEAD ? 1 : 2); ++walk) {
        long long ws = 0;
        for (int n0 = 0; n0 < a.num_seqs; n0 += 32) {
            const int n = n0 + lane;
            long long b = 0, e = 0, slot = 0;
            if (n >= a.num_seqs || !sequence(a, n, b, e, slot, false)) b = e = 0;
            const int chunks = static_cast<int>((e - b + kChunk - 1) / kChunk), segs = (chunks + a.seg - 1) / a.seg;
            const int whole = chunks / a.seg, mine = AHEAD ? max(segs - 1, 0) : walk == 0 ? whole : segs - whole;
            int upto = mine, held = segs > 1 ? segs : 0;
            const int states = held;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int x = __shfl_up_sync(kFullMask, upto, o), y = __shfl_up_sync(kFullMask, held, o);
                if (lane >= o) upto += x, held += y;
            }
            const unsigned hit = __ballot_sync(kFullMask, rank < base + upto);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    const int k = rank - (base + upto - mine) + (walk == 0 ? 0 : whole);
                    u.begin = b + static_cast<long long>(k) * a.seg * kChunk;
                    u.slot = slot;
                    u.ws = ws + held - states;
                    u.chunks = min(a.seg, chunks - k * a.seg);
                    u.len = static_cast<int>(min(e - u.begin, static_cast<long long>(u.chunks) * kChunk));
                    u.k = k;
                    u.parts = segs;
                    // bounds that go back make sequences overlap (the status has it): no state behind the workspace's
                    u.found = segs == 1 || u.ws + segs <= a.ws_states;
                }
                return;
            }
            base += __shfl_sync(kFullMask, upto, 31);
            ws += __shfl_sync(kFullMask, held, 31);
        }
    }
}

template <int P, int S>
__global__ void __launch_bounds__(kChunkNT, 1) ssm_chunk_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SsmMaps maps) {
    using K = ChunkCfg<P, S>;
    constexpr int NB = K::NB, NC = K::NC;
    constexpr bool WB = K::WB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * CK_N];
    __shared__ Unit us;
    __shared__ volatile float head_s[2][3];  // of the unit's heads: A (base 2), dt's bias, D
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t most_polls;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // units: per segment the groups, and in each the pairs of heads (heads of 128: the heads)
    const int in_group = a.H / a.G, per_group = (in_group * P + 127) / 128, per_seg = a.G * per_group;
    const int rank = blockIdx.x / per_seg, which = blockIdx.x % per_seg, g = which / per_group;
    const int h0 = g * in_group + which % per_group * (128 / P), heads = min(128 / P, (g + 1) * in_group - h0);
    if (blockIdx.x == 0)
        for (int n = tid; n < a.num_seqs; n += kChunkNT) {
            long long b, e, slot;
            sequence(a, n, b, e, slot, true);
        }
    if (warp == 0) find_unit<false>(a, rank, us);
    if (tid == 32) {
        for (int i = 0; i < 2 * CK_N; ++i) {
            const int id = i / 2;
            // B and C arrive one after the other; at the others but for the copies' and products' arrive warps
            const int count = id == CK_BC ? 2 : id == CK_YF || id == CK_O || id == CK_XE || id == CK_M ? 16
                              : id == CK_V ? (P == 64 ? 8 : 4)
                              : id == CK_XH || id == CK_S || id == CK_XL ? 8 : 1;
            tc::mbar_init(&bars[i], count);
        }
        most_polls = a.polls;
    }
    __syncthreads();
    if (!us.found) return;
    if (warp == 17) tc::tmem_alloc(&tmem_slot, 512);
    if (tid < 2) {
        const int h = h0 + (tid < heads ? tid : 0);
        head_s[tid][0] = -expf(a.A_log[h]) * 1.44269504f;
        head_s[tid][1] = a.dt_bias[h];
        head_s[tid][2] = a.D ? a.D[h] : 0.f;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot;
    const Unit& u = us;
    uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = tc::smem_u32(sm);

    auto wait = [&](int id, int c) -> bool {
        if (tc::mbar_wait_most<kPolls>(&bars[2 * id + (c & 1)], c >> 1 & 1, &most_polls)) return true;
        most_polls = 0;
        return false;
    };
    auto warp_wait = [&](int id, int c) -> bool {
        const bool ok = __all_sync(kFullMask, wait(id, c));
        tc::fence_after();
        return ok;
    };
    auto one_wait = [&](int id, int c) -> bool {
        const bool ok = wait(id, c);
        tc::fence_after();
        return ok;
    };
    auto warp_arrive = [&](int id, int c) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[2 * id + (c & 1)]);
    };
    auto vec = [&](int c, int hh) { return reinterpret_cast<float*>(sm + K::OFF_V) + ((c & 1) * 2 + hh) * K::VEC; };
    const uint32_t trow = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    auto all_left = [] { asm volatile("bar.sync 1, 640;" ::: "memory"); };  // every role has left its loop

    if (warp >= 16) {
        attn::regs_down<kRegsIssue>();  // by the whole warpgroup, then its warps part
        int nx = 0, nbc = 0, nz = 0;    // loads that this lane has issued: chunks of x, tiles of B and C in turn, chunks of the gate
        if (warp == 16 && attn::elect()) {
            // -------------------------------------------------------- loader
            bool ok = true;
            for (int c = 0; c < u.chunks && ok; ++c) {
                const int row = static_cast<int>(u.begin) + c * kChunk;
                if (c >= 2) ok = wait(CK_XE, c - 2);
                if (!ok) break;
                uint64_t* bar = &bars[2 * CK_X + (c & 1)];
                const int halves = heads * P / 64;
                tc::mbar_expect_tx(bar, halves * 16384);
                for (int i = 0; i < halves; ++i) attn::tma_load_2d(sb + K::OFF_X + (c & 1) * K::X + i * 16384, &maps.x, h0 * P + 64 * i, row, bar);
                ++nx;
                if (c >= NB) ok = wait(CK_UPD, c - NB);
                if (!ok) break;
                bar = &bars[2 * CK_BC + (c & 1)];
                tc::mbar_expect_tx(bar, K::CB);
#pragma unroll
                for (int i = 0; i < S / 64; ++i) attn::tma_load_2d(sb + K::OFF_B + c % NB * K::CB + i * 16384, &maps.B, g * S + 64 * i, row, bar);
                ++nbc;
                if (NB > NC && c >= 1) ok = wait(CK_UPD, c - 1);  // C's own chunk before, the low parts in its place included
                if (!ok) break;
                tc::mbar_expect_tx(bar, K::CB);
#pragma unroll
                for (int i = 0; i < S / 64; ++i) attn::tma_load_2d(sb + K::OFF_C + c % NC * K::CB + i * 16384, &maps.C, g * S + 64 * i, row, bar);
                ++nbc;
                if (NB == 1 && c + 1 < u.chunks) {  // the next ones can start late only: from L2, then (four prompts 353 -> 348 us)
#pragma unroll
                    for (int i = 0; i < S / 64; ++i) {
                        tma_prefetch_2d(&maps.B, g * S + 64 * i, row + kChunk);
                        tma_prefetch_2d(&maps.C, g * S + 64 * i, row + kChunk);
                    }
                }
            }
        }
        // The products' loops are unrolled by four only: unrolled in full, their descriptors, which are the same from chunk to chunk,
        // were kept in more registers than there are.  Two lanes issue: one what the outputs are made of, the other the state's update, so that neither chain waits for the
        // other's barriers.  What must be in order between the two is so by those: a chunk's update ends behind its Y = C S^T, whose operands'
        // places the middle and low parts take, and that behind its G.
        if (warp == 17 && attn::elect()) {
            // -------------------------------------------------------- G, Y
            constexpr uint32_t ID_G = tc::idesc_bf16(128, 128, 0, 0, 0), ID_MX = tc::idesc_bf16(128, P, 0, 1, 0);
            const uint64_t dC = tc::sdesc(sb + K::OFF_C, 16, 1024), dB = tc::sdesc(sb + K::OFF_B, 16, 1024), dS = tc::sdesc(sb + K::OFF_S, 16, 1024);
            const uint64_t dX = tc::sdesc(sb + K::OFF_X, 16384, 1024);
            auto pairs = [&](int c) -> bool {  // G of chunk c
                if (!one_wait(CK_BC, c)) return false;
                const uint64_t off = c % NB * (K::CB >> 4), coff = c % NC * (K::CB >> 4);
#pragma unroll 1
                for (uint32_t q = 0; q < S / 64; ++q)
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) tc::mma_bf16(tm + K::TM_G, dC + coff + q * 1024 + 2 * k, dB + off + q * 1024 + 2 * k, ID_G, q + k > 0);
                tc::commit(&bars[2 * CK_G + (c & 1)]);
                return true;
            };
            bool ok = true;
            for (int c = 0; c < u.chunks && ok; ++c) {
                const uint64_t coff = c % NC * (K::CB >> 4), xoff = (c & 1) * (K::X >> 4);
                ok = (c == 0 || one_wait(CK_YF, c - 1)) && pairs(c) && one_wait(CK_S, c);
                if (!ok) break;
#pragma unroll 1
                for (uint32_t q = 0; q < S / 64; ++q)
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) tc::mma_bf16(tm + K::TM_Y, dC + coff + q * 1024 + 2 * k, dS + q * 1024 + 2 * k, ID_G, q + k > 0);
                tc::commit(&bars[2 * CK_CS + (c & 1)]);
                ok = one_wait(CK_M, c);
                if (!ok) break;
                // M X in the place of G, which all have read
                constexpr int HEADS = 128 / P;
#pragma unroll 1
                for (int h = 0; h < HEADS; ++h) {
                    if (h < heads) {
#pragma unroll 1
                        for (uint32_t q = 0; q < 2; ++q)
#pragma unroll
                            for (uint32_t k = 4 * q, i = 0; i < 4; ++k, ++i)
                                tc::mma_bf16_ts(tm + K::TM_G + 64 * h, tm + K::TM_M + 64 * h + 8 * k, dX + xoff + h * 1024 + k * 128, ID_MX, k > 0);
                    }
                    tc::commit(&bars[2 * (CK_MX0 + h) + (c & 1)]);
                }
            }
            // nothing of this CTA's may be in flight when it ends, its barriers' arrivals included
            tc::commit(&bars[2 * CK_DRAIN]);
            tc::mbar_wait(&bars[2 * CK_DRAIN], 0, kPolls);
        }
        if (warp == 19 && attn::elect()) {
            // -------------------------------------------------------- the gate's rows, and the stores of whole chunks, in one place
            const int halves = heads * P / 64;
            auto gate = [&](int c) {
                uint64_t* bar = &bars[2 * CK_Z + (c & 1)];
                tc::mbar_expect_tx(bar, halves * 3 * K::ZBOX);
                for (int i = 0; i < halves; ++i)
                    for (int j = 0; j < 3; ++j)
                        attn::tma_load_2d(sb + K::OFF_Z + (3 * i + j) * K::ZBOX, &maps.z, h0 * P + 64 * i, static_cast<int>(u.begin) + c * kChunk + 32 + 32 * j, bar);
                ++nz;
            };
            bool ok = true;
            if (a.z) gate(0);
            for (int c = 0; c < u.chunks && ok; ++c) {
                ok = wait(CK_O, c);
                if (!ok) break;
                if (u.len - c * kChunk >= kChunk) {
                    for (int i = 0; i < halves; ++i)
                        for (int j = 0; j < 3; ++j)
                            tma_store_2d(&maps.y, h0 * P + 64 * i, static_cast<int>(u.begin) + c * kChunk + 32 + 32 * j, sb + K::OFF_Z + (3 * i + j) * K::ZBOX);
                    tc::bulk_commit();
                    tc::bulk_wait_read();
                }
                if (!a.z) tc::mbar_arrive(&bars[2 * CK_ZE + (c & 1)]);
                else if (c + 1 < u.chunks) gate(c + 1);
            }
            tc::bulk_wait_all();
        }
        if (warp == 18 && attn::elect()) {
            // -------------------------------------------------------- the state
            constexpr uint32_t ID_UPD = tc::idesc_bf16(128, S, 1, 1, 0);
            const uint64_t dBm = tc::sdesc(sb + K::OFF_B, 16384, 1024), dX = tc::sdesc(sb + K::OFF_X, 16384, 1024);
            const uint64_t dH = tc::sdesc(sb + K::OFF_H, 16384, 1024), dM = tc::sdesc(sb + K::OFF_M, 16384, 1024), dL = tc::sdesc(sb + K::OFF_L, 16384, 1024);
            bool ok = true;
            for (int c = 0; c < u.chunks && ok; ++c) {
                const uint64_t off = WB ? (c & 1) * (K::X >> 4) : c % NB * (K::CB >> 4);
                auto update = [&](uint64_t part, uint32_t k) {
                    tc::mma_bf16(tm + K::TM_S, (WB ? dX + off : part) + k * 128, (WB ? part : dBm + off) + k * 128, ID_UPD, 1);
                };
                ok = one_wait(CK_BC, c) && one_wait(CK_XH, c) && one_wait(CK_S, c);
                if (!ok) break;
#pragma unroll 1
                for (uint32_t q = 0; q < 2; ++q)
#pragma unroll
                    for (uint32_t k = 4 * q, i = 0; i < 4; ++k, ++i) update(dH, k);
                tc::commit(&bars[2 * CK_UPH + (c & 1)]);
                ok = one_wait(CK_XL, c);
                if (!ok) break;
#pragma unroll 1
                for (uint32_t q = 0; q < 4; ++q)
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) update(q < 2 ? dM : dL, (4 * q + i) & 7);
                tc::commit(&bars[2 * CK_UPD + (c & 1)]);
            }
            tc::commit(&bars[2 * CK_DRAIN + 1]);
            tc::mbar_wait(&bars[2 * CK_DRAIN + 1], 0, kPolls);
        }
        __syncwarp();
        all_left();
        if (most_polls == 0) {  // gave up: the copies that nobody waited for land before the CTA ends
            auto land = [&](int id, int n) {
                for (int c = max(n - 2, 0); c < n; ++c) tc::mbar_wait(&bars[2 * id + (c & 1)], c >> 1 & 1, kPolls);
            };
            if (nbc & 1) tc::mbar_arrive(&bars[2 * CK_BC + (nbc >> 1 & 1)]);  // in the place of the last B's C, which nobody expects any more
            land(CK_X, nx);
            land(CK_BC, (nbc + 1) / 2);
            land(CK_Z, nz);
        }
    } else {
        // ------------------------------------------------------------ workers: warpgroups 0, 1 (A) and 2, 3 (B)
        attn::regs_up<kRegsWork>();
        const int wg = warp >> 2, w = warp & 3, t = tid & 127, side = wg & 1;
        const bool isb = wg >= 2;
        const int hh = P == 64 ? side : 0;
        const bool valid = hh < heads;
        const int h = h0 + (valid ? hh : 0);

        // ---- what all do: the weights of pairs in M, the output
        // blocks of 32 columns of M: an A warp has the diagonal one (and the one ahead of it), a B warp those further ahead
        auto mine = [&](int j) {
            if (P == 64) return isb ? j <= w - 2 : j >= w - 1;
            return j == w - wg;
        };
        const uint32_t tM = trow + K::TM_M + (P == 64 ? side * 64 : 0), tY = side * 64 + (wg >> 1) * 32;
        auto weights = [&](int c) -> bool {
            const float* V = vec(c, hh);
            const float pre = V[t];
            if (w - wg < 0 && P == 128) return true;
            if (P == 64 && isb && w < 2) return true;
            if (!warp_wait(CK_G, c)) return false;
            float ahead = pre;  // the decay from the end of block j to the row
#pragma unroll 1
            for (int j = w; j >= 0; --j) {  // one body for all blocks: unrolled, the code did not stay in the instruction cache
                if (j < w - 1) ahead += V[3 * kChunk + j + 1];
                if (!mine(j)) continue;
                const float r = ex2(ahead);
                const attn::f32x2 pp = attn::pair(pre, pre), minus = attn::pair(-1.f, -1.f), rr = attn::pair(r, r);
#pragma unroll
                for (int i0 = 0; i0 < 32; i0 += 16) {
                    float x[16];
                    uint32_t m[8];
                    tc::ld16(trow + K::TM_G + 32 * j + i0, x);
                    tc::wait_ld();
                    const float* Vc = V + 32 * j + i0;
                    if (j == w) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 p = *reinterpret_cast<const float4*>(Vc + i), d = *reinterpret_cast<const float4*>(Vc + 2 * kChunk + i);
                            float f[4], e[4];
                            attn::unpair(attn::fma2(attn::pair(p.x, p.y), minus, pp), f);
                            attn::unpair(attn::fma2(attn::pair(p.z, p.w), minus, pp), f + 2);
                            // dt times its decay first: times G it may leave the range
                            attn::unpair(attn::mul2(attn::pair(ex2(f[0]), ex2(f[1])), attn::pair(d.x, d.y)), e);
                            attn::unpair(attn::mul2(attn::pair(ex2(f[2]), ex2(f[3])), attn::pair(d.z, d.w)), e + 2);
#pragma unroll
                            for (int q = 0; q < 4; ++q) x[i + q] = i0 + i + q <= lane ? e[q] * x[i + q] : 0.f;
                            m[i / 2] = pack_weights(x[i], x[i + 1]);
                            m[i / 2 + 1] = pack_weights(x[i + 2], x[i + 3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(Vc + kChunk + i);
                            float y[4];
                            attn::unpair(attn::mul2(attn::mul2(attn::pair(f.x, f.y), rr), attn::pair(x[i], x[i + 1])), y);
                            attn::unpair(attn::mul2(attn::mul2(attn::pair(f.z, f.w), rr), attn::pair(x[i + 2], x[i + 3])), y + 2);
                            m[i / 2] = pack_weights(y[0], y[1]);
                            m[i / 2 + 1] = pack_weights(y[2], y[3]);
                        }
                    }
                    st8(tM + 16 * j + i0 / 2, m);
                }
            }
            return true;
        };
        const long long col = static_cast<long long>(h0) * P + side * 64;  // the first feature of this half of the tile
        const uint32_t line = static_cast<uint32_t>(side * 16384 + t * 128);  // this row of that half
        // The gate comes by TMA and a whole chunk goes out by TMA, from the same place, but for the first block of rows: a thread's own
        // 64 bytes of a row of global memory, 32 lines per instruction, hold up all that goes through the load and store unit.
        auto output = [&](int c) -> bool {
            const bool live = t < u.len - c * kChunk && valid, staged = w > 0 && u.len - c * kChunk >= kChunk;
            const long long tok = u.begin + c * kChunk + t;
            const uint32_t zt = sb + K::OFF_Z + (3 * side + w - 1) * K::ZBOX + lane * 128;
            uint4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = make_uint4(0, 0, 0, 0);
            if (a.z && w == 0 && live) {
                const uint4* src = reinterpret_cast<const uint4*>(a.z + tok * a.z_stride + col) + (wg >> 1) * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = __ldg(src + i);
            }
            __syncwarp();
            if (!warp_wait(P == 64 ? CK_MX0 + side : CK_MX0, c) || !warp_wait(CK_X, c)) return false;
            if (a.z) {
                if (!warp_wait(CK_Z, c)) return false;
                if (w > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = attn::lds128(zt + ((((wg >> 1) * 4 + i) ^ (lane & 7)) << 4));
                }
            } else if (c > 0 && !warp_wait(CK_ZE, c - 1)) {
                return false;
            }
            const uint32_t at = sb + K::OFF_X + (c & 1) * K::X + line;
            const int t7 = anew(t) & 7;
            const float* V = vec(c, hh);
            float sum = V[t];  // the decay from the chunk's start
            for (int j = 0; j < w; ++j) sum += V[3 * kChunk + j];
            const float D = head_s[hh][2], from = ex2(sum);
            const attn::f32x2 dd = attn::pair(D, D), ff = attn::pair(from, from);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s[16], y[16];
                tc::ld16(trow + K::TM_Y + tY + 16 * i, s);
                tc::ld16(trow + K::TM_G + tY + 16 * i, y);
                tc::wait_ld();
                if (i == 1) {
                    tc::fence_before();
                    warp_arrive(CK_YF, c);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 x = attn::lds128(at + ((((wg >> 1) * 4 + 2 * i + q) ^ t7) << 4));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z[2 * i + q].x, z[2 * i + q].y, z[2 * i + q].z, z[2 * i + q].w};
                    uint32_t r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = 8 * q + 2 * k;
                        attn::f32x2 o = attn::fma2(attn::widen2(xs[k]), dd, attn::fma2(ff, attn::pair(s[j], s[j + 1]), attn::pair(y[j], y[j + 1])));
                        if (a.z) o = attn::mul2(o, attn::silu2(attn::widen2(zs[k])));
                        float f[2];
                        attn::unpair(o, f);
                        r[k] = pack_bf16x2(f[0], f[1]);
                    }
                    z[2 * i + q] = make_uint4(r[0], r[1], r[2], r[3]);
                }
            }
            warp_arrive(CK_XE, c);
            uint4* dst = reinterpret_cast<uint4*>(a.out + tok * a.H * P + col) + (wg >> 1) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (staged) attn::sts128(zt + ((((wg >> 1) * 4 + i) ^ (lane & 7)) << 4), z[i]);
                else if (live) dst[i] = z[i];
            }
            tc::fence_proxy_async();
            warp_arrive(CK_O, c);
            return true;
        };

        // ---- what B does besides: dt and the decays' sums, X', the state between two chunks (thread = feature)
        const int ph = P == 64 ? t >> 6 : 0;  // this feature's head
        const bool there = ph < heads;
        auto srow = [&] { return (static_cast<long long>(h0 + (there ? ph : 0)) * P + (P == 64 ? t & 63 : t)) * S + side * (S / 2); };
        auto state = [&] { return static_cast<long long>(a.H) * P * S; };
        bool ok = true;
        if (isb) {  // the unit's first state: the pool's (for the first of several segments its copy), or what the segments ahead add up to
            const float* src = (u.parts == 1 ? a.state + u.slot * state() : a.ws + u.ws * state()) + srow();
            // The first segment's copy is there if its own state is.  (The same for all of the CTA's heads, which one CTA ahead has.)
            if (u.k == 0 && u.parts > 1) ok = a.ws_decay[(u.ws + 1) * a.H + h0] != kNoState;
            float s[S / 2];
#pragma unroll
            for (int q = 0; q < S / 2; q += 8) {
                if (there && u.k == 0) {
                    ld_state(src + q, s + q);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[q + i] = 0.f;
                }
            }
            for (int j = 0; j < u.k; ++j) {
                const long long at = u.ws + 1 + j;
                const float decay = a.ws_decay[at * a.H + h0 + (there ? ph : 0)], f = ex2(decay);
                ok = ok && decay != kNoState;
                if (!there) continue;
                const float* from = a.ws + at * state() + srow();
#pragma unroll
                for (int q = 0; q < S / 2; q += 8) {
                    float v[8];
                    ld_state(from + q, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[q + i] = fmaf(f, s[q + i], v[i]);
                }
            }
            if (!ok) most_polls = 0;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S / 32; ++i) {
                float v[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) v[q] = s[16 * i + q];
                tc::st16(trow + K::TM_S + side * (S / 2) + 16 * i, v);
            }
            tc::wait_st();
        }
        // dt and the decays' sums of chunk c, a block of 32 tokens each by the warps of M's first two blocks of rows, which have the least of it
        const bool sums = w < 2 && (P == 64 || side == 0);
        const int block = (isb ? 2 : 0) + w;
        auto raw_at = [&](int c) {
            const int i = c * kChunk + block * 32 + lane;
            return sums && valid && i < u.len ? a.dt[(u.begin + i) * a.dt_stride + h] : static_cast<uint16_t>(0);
        };
        uint16_t raw = raw_at(0);
        auto decays = [&](int c) {
            float* V = vec(c, hh);
            const int i = block * 32 + lane;
            const float dt = valid && i < u.len - c * kChunk ? softplus(bf16_to_f32(raw) + head_s[hh][1]) : 0.f;
            raw = raw_at(c + 1);
            const float step = log_decay(head_s[hh][0], dt);
            float upto = step, behind = __shfl_down_sync(kFullMask, step, 1);
            if (lane == 31) behind = 0.f;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const float x = __shfl_up_sync(kFullMask, upto, o), y = __shfl_down_sync(kFullMask, behind, o);
                if (lane >= o) upto += x;
                if (lane + o < 32) behind += y;
            }
            V[i] = upto;
            V[kChunk + i] = dt * ex2(behind);
            V[2 * kChunk + i] = dt;
            if (lane == 31) V[3 * kChunk + block] = upto;
            warp_arrive(CK_V, c);
        };
        // this token's weight in the state behind the chunk
        auto weight_of = [&](int c) {
            const float* V = vec(c, hh);
            float behind = 0.f;
            for (int j = w + 1; j < 4; ++j) behind += V[3 * kChunk + j];
            return V[kChunk + t] * ex2(behind);
        };
        // The row (of x, or of B) times its weight, as bf16 high parts or as the two parts of what they leave.  In fp32: packed bf16 products took twice the time.
        auto weigh = [&](int c, float weight, bool high) {
            const attn::f32x2 ww = attn::pair(weight, weight), minus = attn::pair(-1.f, -1.f);
            const int t7 = anew(t) & 7;
            const uint32_t from = sb + (WB ? K::OFF_B + c % NB * K::CB : K::OFF_X + (c & 1) * K::X), row = WB ? t * 128 : line;
#pragma unroll
            for (int q0 = WB ? side * 4 : 0, n = 0; n < (WB ? 1 : 2); q0 += 4, ++n) {
                uint4 x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = attn::lds128(from + row + (((q0 + q) ^ t7) << 4));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[4] = {x[q].x, x[q].y, x[q].z, x[q].w}, l[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        attn::f32x2 p = attn::mul2(attn::widen2(v[k]), ww);
                        v[k] = pack_part<WB>(p);
                        if (!high) {
                            p = attn::fma2(attn::widen2(v[k]), minus, p);
                            v[k] = pack_part<WB>(p);
                            l[k] = pack_part<WB>(attn::fma2(attn::widen2(v[k]), minus, p));
                        }
                    }
                    const uint32_t at = sb + row + (((q0 + q) ^ t7) << 4);
                    attn::sts128(at + (high ? K::OFF_H : K::OFF_M), make_uint4(v[0], v[1], v[2], v[3]));
                    if (!high) attn::sts128(at + K::OFF_L, make_uint4(l[0], l[1], l[2], l[3]));
                }
            }
            tc::fence_proxy_async();
        };
        // A: X' of chunk c, high parts
        auto high_parts = [&](int c) -> bool {
            const int rows = min(kChunk, u.len - c * kChunk);
            if (!warp_wait(CK_X, c) || !warp_wait(CK_V, c)) return false;
            if (WB && !warp_wait(CK_BC, c)) return false;
            if (rows < kChunk || !valid) {  // what a weight of zero meets must be finite: rows behind the sequence may hold anything
                if (!WB && !warp_wait(CK_BC, c)) return false;
                const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (t >= rows || !valid) attn::sts128(sb + K::OFF_X + (c & 1) * K::X + line + (q << 4), none);
                    // of B: this thread's half of the row
                    if (t >= rows && (S == 128 || (q ^ t & 7) >> 2 == side)) attn::sts128(sb + K::OFF_B + c % NB * K::CB + (S == 128 ? line : t * 128) + (q << 4), none);
                }
            }
            if (c > 0 && !warp_wait(CK_UPH, c - 1)) return false;
            weigh(c, weight_of(c), true);
            warp_arrive(CK_XH, c);
            return true;
        };
        float weight = 0.f;
        // B: the state that chunk c begins with: a copy in bf16 for Y, and the decayed state
        auto begin = [&](int c) -> bool {
            if (!warp_wait(CK_V, c)) return false;
            weight = weight_of(c);
            const float* W = vec(c, ph) + 3 * kChunk;  // of this feature's head
            const float keep = ex2((W[0] + W[1]) + (W[2] + W[3]));
            if (c > 0 && !warp_wait(CK_UPD, c - 1)) return false;
            const attn::f32x2 kk = attn::pair(keep, keep);
            const int ts = anew(t);
#pragma unroll
            for (int i = 0; i < S / 32; ++i) {
                float s[16];
                const int n0 = side * (S / 2) + 16 * i;
                tc::ld16(trow + K::TM_S + n0, s);
                tc::wait_ld();
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    attn::sts128(sb + K::OFF_S + tc::sw_chunk(ts, n0 / 8 + q, 128),
                                 make_uint4(pack_bf16x2(s[8 * q], s[8 * q + 1]), pack_bf16x2(s[8 * q + 2], s[8 * q + 3]), pack_bf16x2(s[8 * q + 4], s[8 * q + 5]),
                                            pack_bf16x2(s[8 * q + 6], s[8 * q + 7])));
#pragma unroll
                for (int q = 0; q < 16; q += 2) attn::unpair(attn::mul2(attn::pair(s[q], s[q + 1]), kk), s + q);
                tc::st16(trow + K::TM_S + n0, s);
            }
            tc::wait_st();
            tc::fence_before();
            tc::fence_proxy_async();
            warp_arrive(CK_S, c);
            return true;
        };
        if (!isb) {
            for (int j = w + 1; j < 4; ++j) {  // tokens behind the row's: zero, once for all
                const uint32_t zero[16] = {};
                if (P == 64 || wg == 0) attn::tm_st16(tM + 16 * j, zero);
            }
        }
        if (sums) decays(0);
#pragma unroll 1
        for (int c = -1; ok && c < u.chunks; ++c) {
            if (c >= 0) {
                ok = (isb || warp_wait(CK_V, c)) && weights(c);
                if (!ok) break;
                tc::wait_st();
                tc::fence_before();
                warp_arrive(CK_M, c);
                // The sums of c + 1 go where those of c - 1 were: what is waited for here (B) or for the weights (A) stands behind the last
                // reading of those, in the output of c - 1.
                if (isb) {  // once the state's copy and C have been read their places are those of the other parts of X'
                    ok = warp_wait(CK_CS, c) && warp_wait(CK_X, c);
                    if (!ok) break;
                    if (sums && c + 1 < u.chunks) decays(c + 1);
                    ok = warp_wait(CK_XH, c);
                    if (!ok) break;
                    weigh(c, weight, false);
                    warp_arrive(CK_XL, c);
                }
                if (!isb && sums && c + 1 < u.chunks) decays(c + 1);
            }
            if (c + 1 < u.chunks) {
                ok = isb ? begin(c + 1) : high_parts(c + 1);
            }
            if (c >= 0) ok = ok && output(c);
        }
        if (ok && isb) warp_wait(CK_UPD, u.chunks - 1);
        __syncwarp();
        all_left();
        if (isb && most_polls != 0 && u.k == u.parts - 1) {
            float* dst = a.state + u.slot * state() + srow();
#pragma unroll 1
            for (int i = 0; i < S / 32; ++i) {
                float v[16];
                tc::ld16(trow + K::TM_S + side * (S / 2) + 16 * i, v);
                tc::wait_ld();
                if (there) st_state(dst + 16 * i, v), st_state(dst + 16 * i + 8, v + 8);
                __syncwarp();
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 17) tc::tmem_dealloc(tm, 512);
    if (tid == 0 && most_polls == 0) atomicOr(a.status, kStatusTimeout);
}

// The states that the segments ahead end in, each from a zero state (the first of a sequence from the pool's, of which it also leaves a
// copy), and the logarithms of their decays (kNoState: gave up).  A token's weight is its decay to the segment's end, so nothing is carried from chunk to
// chunk: the chunks are taken from the last to the first with the sum of the steps behind them, and sixteen warps make X' of one
// (high parts in x's own tile, middle ones beside it, low ones in the other stage's place for those) while the products of the one before run.
template <int P, int S>
struct AheadCfg {
    static constexpr bool WB = ChunkCfg<P, S>::WB;
    // x, its middle parts, B, with x's high parts in its own place and the low ones in that of the other stage's middle ones; or x, B, B's middle and
    // low parts, with its high ones in its own place.
    static constexpr uint32_t X = 32768, CB = kChunk * S * 2, STAGE = WB ? X + 3 * CB : 2 * X + CB;
    static constexpr uint32_t OFF_B = WB ? X : 2 * X, OFF_H = WB ? X : 0, OFF_M = WB ? X + CB : X, OFF_L = WB ? X + 2 * CB : X;
    static constexpr uint32_t SMEM = 2 * STAGE + 1024;
};
constexpr int kAheadNT = 576;

template <int P, int S>
__global__ void __launch_bounds__(kAheadNT, 1) ssm_ahead_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SsmMaps maps) {
    using K = AheadCfg<P, S>;
    constexpr bool WB = K::WB;
    constexpr int BATCH = kSegment;  // chunks whose weights are made at once: a segment ahead is whole, a number of batches
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[2], ready[2], done[2], drain;
    __shared__ Unit us;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t most_polls;
    __shared__ alignas(16) float weight_s[2][2][BATCH * kChunk], block_s[2][2][BATCH * 4];  // block_s is read four at a time
    __shared__ float total_s[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int in_group = a.H / a.G, per_group = (in_group * P + 127) / 128, per_seg = a.G * per_group;
    const int which = blockIdx.x % per_seg, g = which / per_group;
    const int h0 = g * in_group + which % per_group * (128 / P), heads = min(128 / P, (g + 1) * in_group - h0);
    if (warp == 0) find_unit<true>(a, blockIdx.x / per_seg, us);
    if (tid == 32) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&ready[i], 16);
            tc::mbar_init(&done[i], 1);
        }
        tc::mbar_init(&drain, 1);
        most_polls = a.polls;
    }
    __syncthreads();
    if (!us.found) return;
    if (warp == 17) tc::tmem_alloc(&tmem_slot, 128);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot;
    const Unit& u = us;
    const uint32_t sb = tc::smem_u32(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
    // i: the number of a chunk from the segment's end
    auto wait = [&](uint64_t* bars, int i) -> bool {
        if (tc::mbar_wait_most<kPolls>(&bars[i & 1], i >> 1 & 1, &most_polls)) return true;
        most_polls = 0;
        return false;
    };

    if (warp == 16) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            int i = 0;
            for (; i < u.chunks; ++i) {
                if (i >= 2 && !wait(done, i - 2)) break;
                const int row = static_cast<int>(u.begin) + (u.chunks - 1 - i) * kChunk, halves = heads * P / 64;
                const uint32_t to = sb + (i & 1) * K::STAGE;
                tc::mbar_expect_tx(&full[i & 1], halves * 16384 + K::CB);
                for (int j = 0; j < halves; ++j) attn::tma_load_2d(to + j * 16384, &maps.x, h0 * P + 64 * j, row, &full[i & 1]);
#pragma unroll
                for (int j = 0; j < S / 64; ++j) attn::tma_load_2d(to + K::OFF_B + j * 16384, &maps.B, g * S + 64 * j, row, &full[i & 1]);
            }
            for (int j = max(i - 2, 0); j < i; ++j) tc::mbar_wait(&full[j & 1], j >> 1 & 1, kPolls);  // where others gave up nobody else does
        }
    } else if (warp == 17) {
        // ------------------------------------------------------------ MMA issue
        if (attn::elect()) {
            constexpr uint32_t ID = tc::idesc_bf16(128, S, 1, 1, 0);
            const uint64_t dX = tc::sdesc(sb, 16384, 1024);
            for (int i = 0; i < u.chunks; ++i) {
                if (!wait(full, i) || !wait(ready, i)) break;
                tc::fence_after();
                const uint64_t stage = dX + (i & 1) * (K::STAGE >> 4), low = (WB ? stage : dX + (~i & 1) * (K::STAGE >> 4)) + (K::OFF_L >> 4);
#pragma unroll 1
                for (uint32_t q = 0; q < 6; ++q)
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t k = (4 * q + j) & 7;
                        const uint64_t part = (q < 2 ? stage + (K::OFF_H >> 4) : q < 4 ? stage + (K::OFF_M >> 4) : low) + k * 128;
                        tc::mma_bf16(tm, WB ? stage + k * 128 : part, WB ? part : stage + (K::OFF_B >> 4) + k * 128, ID, i + q + j > 0);
                    }
                tc::commit(&done[i & 1]);
            }
            // nothing of this CTA's may be in flight when it ends, its barriers' arrivals included
            tc::commit(&drain);
            tc::mbar_wait(&drain, 0, kPolls);
        }
    } else {
        // ------------------------------------------------------------ workers: a token's 32 features, then a quarter of a feature's state
        const int wg = warp >> 2, w = warp & 3, t = tid & 127, side = wg & 1, hh = P == 64 ? side : 0;
        const bool valid = hh < heads;
        // the weights of a batch within blocks of 32 tokens, and the blocks' sums; blocks count from the batch's first token on
        auto weights = [&](int batch) {
            const int first = u.chunks - (batch + 1) * BATCH, head = warp & 1;
            if (head >= heads) return;
            const float A = -expf(a.A_log[h0 + head]) * 1.44269504f, bias = a.dt_bias[h0 + head];
            float dt[BATCH / 2];
#pragma unroll
            for (int j = 0; j < BATCH / 2; ++j) {
                const int b = 8 * j + (warp >> 1);
                dt[j] = bf16_to_f32(a.dt[(u.begin + first * kChunk + b * 32 + lane) * a.dt_stride + h0 + head]);
            }
#pragma unroll
            for (int j = 0; j < BATCH / 2; ++j) {
                const int b = 8 * j + (warp >> 1);
                const float d = softplus(dt[j] + bias), step = log_decay(A, d);
                float behind = __shfl_down_sync(kFullMask, step, 1);
                if (lane == 31) behind = 0.f;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const float y = __shfl_down_sync(kFullMask, behind, o);
                    if (lane + o < 32) behind += y;
                }
                weight_s[batch & 1][head][b * 32 + lane] = d * ex2(behind);
                if (lane == 0) block_s[batch & 1][head][b] = behind + step;
            }
        };
        auto together = [] { asm volatile("bar.sync 1, 512;" ::: "memory"); };
        weights(0);
        together();
        float gone = 0.f;  // the steps behind the chunk
        bool ok = true;
        for (int i = 0; i < u.chunks; ++i) {
            const int batch = i / BATCH;
            if (i % BATCH == 0 && i + BATCH < u.chunks) weights(batch + 1);
            if (ok) {
                ok = __all_sync(kFullMask, wait(full, i));
            }
            if (ok) {
                const int c = BATCH - 1 - i % BATCH;  // in the batch
                float weight = 0.f;
                if (valid) {
                    const float4 sums = *reinterpret_cast<const float4*>(&block_s[batch & 1][hh][4 * c]);
                    const float behind = w == 0 ? sums.y + sums.z + sums.w : w == 1 ? sums.z + sums.w : w == 2 ? sums.w : 0.f;
                    weight = weight_s[batch & 1][hh][c * kChunk + t] * ex2(gone + behind);
                    gone += (sums.x + sums.y) + (sums.z + sums.w);
                }
                const attn::f32x2 ww = attn::pair(weight, weight), minus = attn::pair(-1.f, -1.f);
                constexpr int NQ = WB ? 2 : 4;  // pieces of 16 bytes: of half a row of x, of a quarter of B's
                const int q0 = WB ? wg * 2 : (wg >> 1) * 4;
                const uint32_t line = sb + (WB ? 0 : side * 16384) + t * 128, tile = line + (i & 1) * K::STAGE;
                uint4 x[NQ], low[NQ];
#pragma unroll
                for (int q = 0; q < NQ; ++q) x[q] = valid ? attn::lds128(tile + K::OFF_H + (((q0 + q) ^ (t & 7)) << 4)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    uint32_t v[4] = {x[q].x, x[q].y, x[q].z, x[q].w}, l[4], r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        attn::f32x2 p = attn::mul2(attn::widen2(v[k]), ww);
                        v[k] = pack_part<WB>(p);
                        p = attn::fma2(attn::widen2(v[k]), minus, p);
                        l[k] = pack_part<WB>(p);
                        r[k] = pack_part<WB>(attn::fma2(attn::widen2(l[k]), minus, p));
                    }
                    attn::sts128(tile + K::OFF_H + (((q0 + q) ^ (t & 7)) << 4), make_uint4(v[0], v[1], v[2], v[3]));
                    x[q] = make_uint4(l[0], l[1], l[2], l[3]);
                    low[q] = make_uint4(r[0], r[1], r[2], r[3]);
                }
                // The products of the chunk before have its middle parts and, in the place of this one's, its low parts.
                if (!WB && i > 0) ok = __all_sync(kFullMask, wait(done, i - 1));
                if (ok) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const uint32_t at = ((q0 + q) ^ (t & 7)) << 4;
                        attn::sts128(tile + K::OFF_M + at, x[q]);
                        attn::sts128((WB ? tile : line + (~i & 1) * K::STAGE) + K::OFF_L + at, low[q]);
                    }
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&ready[i & 1]);
                }
            }
            if (i % BATCH == BATCH - 1) together();  // all warps come here, those that gave up too
        }
        if (w == 0 && wg < heads && lane == 0 && P == 64) total_s[wg] = gone;
        if (P == 128 && tid == 0) total_s[0] = gone;
        together();
        ok = ok && __all_sync(kFullMask, wait(done, u.chunks - 1));
        tc::fence_after();
        if (ok) {
            const int ph = P == 64 ? t >> 6 : 0;
            const bool there = ph < heads;
            const long long state = static_cast<long long>(a.H) * P * S;
            const long long row = (static_cast<long long>(h0 + (there ? ph : 0)) * P + (P == 64 ? t & 63 : t)) * S + wg * (S / 4);
            const float total = total_s[there ? ph : 0], f = ex2(total);
            if (wg == 0 && there && (P == 64 ? t & 63 : t) == 0) a.ws_decay[(u.ws + 1 + u.k) * a.H + h0 + ph] = total;
#pragma unroll
            for (int i = 0; i < S / 64; ++i) {
                float v[16];
                tc::ld16(tm + (static_cast<uint32_t>(w * 32) << 16) + wg * (S / 4) + 16 * i, v);
                tc::wait_ld();
                if (there) {
                    if (u.k == 0) {  // the pool's state, copied too: the last segment may have replaced it when the first one starts
#pragma unroll
                        for (int q = 0; q < 16; q += 8) {
                            float x[8];
                            ld_state(a.state + u.slot * state + row + 16 * i + q, x);
                            st_state(a.ws + u.ws * state + row + 16 * i + q, x);
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[q + k] = fmaf(x[k], f, v[q + k]);
                        }
                    }
                    float* dst = a.ws + (u.ws + 1 + u.k) * state + row + 16 * i;
                    st_state(dst, v);
                    st_state(dst + 8, v + 8);
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 17) tc::tmem_dealloc(tm, 128);
    if (tid == 0 && most_polls == 0) {
        for (int i = 0; i < heads; ++i) a.ws_decay[(u.ws + 1 + u.k) * a.H + h0 + i] = kNoState;
        atomicOr(a.status, kStatusTimeout);
    }
}

}  // namespace ssm
}  // namespace gdn
