// tile_util.cuh -- what the tile kernels (attn_tiles.cuh, ssm_chunk.cuh) share: TMEM rows of 32 columns, pairs of fp32
// operations in one instruction, the election of a lane, registers
// moved between warpgroups.
#pragma once

#include "attn_mma.cuh"
#include "common.cuh"

namespace gdn {
namespace attn {

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
// Two packed bf16 as a pair of fp32.
__device__ __forceinline__ f32x2 widen2(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
// z / (1 + e^-z) of both.  Beyond the range of e^-z its reciprocal is 0, as the quotient is.
__device__ __forceinline__ f32x2 silu2(f32x2 z) {
    float e[2], r[2];
    unpair(mul2(z, pair(-1.44269504f, -1.44269504f)), e);
    unpair(add2(pair(fast_exp2(e[0]), fast_exp2(e[1])), pair(1.f, 1.f)), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(e[0]));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(e[1]));
    return mul2(z, pair(r[0], r[1]));
}
// The same as z e^z / (1 + e^z) with one reciprocal, of the denominators' product, for where exponentials and reciprocals are many (convolution of
// 23508 tokens of 8192 channels: 141 us, 143 with the form above; the scan's gate in four prompts: 339 us, 333 with the form above).
// e^z is held at e^40, whose square is still a number: from there on the quotient rounds to 1.  z comes last: times e^40 a z of 2^71 and more
// would leave the range.
__device__ __forceinline__ f32x2 silu2_joint(f32x2 z) {
    float e[2], r;
    unpair(mul2(z, pair(1.44269504f, 1.44269504f)), e);
    const f32x2 t = pair(fast_exp2(fminf(e[0], 57.7f)), fast_exp2(fminf(e[1], 57.7f)));
    unpair(add2(t, pair(1.f, 1.f)), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e[0] * e[1]));
    return mul2(z, mul2(mul2(t, pair(e[1], e[0])), pair(r, r)));
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(one));
    return one != 0;
}
// A warpgroup takes more registers per thread, or gives some up.
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

}  // namespace attn
}  // namespace gdn
