// ssm.cu -- launch of the state space scan (ssm.cuh, ssm_chunk.cuh).
#include <algorithm>
#include <atomic>
#include <cstring>

#include "host.h"
#include "launch.h"
#include "ssm_chunk.cuh"

namespace gdn {
namespace {

// Tokens as rows of `width` elements: boxes of 64 columns and `rows` rows, 128-byte swizzle, zero fill outside.
bool encode_tokens(CUtensorMap* map, const void* base, long long T, long long width, long long stride, unsigned rows = 128) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, rows}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int P, int S>
cudaError_t run(const SsmArgs& a, const SsmMaps& maps, unsigned grid, cudaStream_t stream) {
    using C = ssm::ChunkCfg<P, S>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = raise_smem(ssm::ssm_chunk_kernel<P, S>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    // the split of registers among roles waits forever where the launch has fewer than it adds up to
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, ssm::ssm_chunk_kernel<P, S>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < ssm::kRegsLaunch) return cudaErrorInvalidConfiguration;
    ssm::ssm_chunk_kernel<P, S><<<grid, ssm::kChunkNT, C::SMEM, stream>>>(a, maps);
    return cudaGetLastError();
}

template <int P, int S>
cudaError_t ahead(const SsmArgs& a, const SsmMaps& maps, unsigned grid, cudaStream_t stream) {
    using C = ssm::AheadCfg<P, S>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = raise_smem(ssm::ssm_ahead_kernel<P, S>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    ssm::ssm_ahead_kernel<P, S><<<grid, ssm::kAheadNT, C::SMEM, stream>>>(a, maps);
    return cudaGetLastError();
}

template <int P, int S>
cudaError_t chunks(SsmArgs a, long long max_len, void* workspace, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    SsmMaps maps;
    const long long inner = static_cast<long long>(a.H) * P, gs = static_cast<long long>(a.G) * S;
    if (!encode_tokens(&maps.x, a.x, a.T, inner, a.x_stride) || !encode_tokens(&maps.B, a.B, a.T, gs, a.b_stride) ||
        !encode_tokens(&maps.C, a.C, a.T, gs, a.c_stride) || !encode_tokens(&maps.y, a.out, a.T, inner, inner, 32) ||
        !encode_tokens(&maps.z, a.z ? a.z : a.x, a.T, inner, a.z ? a.z_stride : a.x_stride, 32))
        return cudaErrorInvalidValue;
    // Segments.  In chunk times of one SM: `share` is the work over the SMs, a chain takes as long as it is, units that are
    // more than the SMs end unevenly by about half a unit, the launch ahead costs two fifths of what it covers, its uneven end
    // included, and a start, and a segment starts from as many states as there are segments ahead, a third of a chunk time each where all SMs read
    // (N = 128), a quarter else.  Measured, us: four prompts of 64, 43, 22 and 56 chunks and 32 units each: 348 whole, 381 to 449 in segments of 8
    // to 48; one of 128 chunks, N = 64: 479 whole, 260, 221, 293, 220, 242, 283, 367 in segments of 8, 16, .. 48, 64; N = 128, one of 192: 930
    // whole, 633, 455, 416, 508, 467, 391, 481; of 256: 1237 whole, 818, 623, 602, 542, 616, 725, 510; of 512: 2459 whole, 2310, 1237,
    // 1082, 1076, 987, 1105, 1008, and 989 in segments of 128.
    const long long per_seg = static_cast<long long>(a.G) * ((a.H / a.G * P + 127) / 128);
    const double total = static_cast<double>((a.T + 127) / 128), share = total * per_seg / sms;
    const double longest = static_cast<double>((std::min(std::max(max_len, 1LL), a.T) + 127) / 128);
    auto cost = [&](double seg) {
        const double parts = std::max(1.0, static_cast<double>(static_cast<long long>((longest + seg - 1) / seg))), units = total / longest * parts * per_seg;
        const double start = seg < longest ? 0.4 * share * (longest - seg) / longest + 3.0 : 0.0, states = (parts - 1) * S / 128;
        return (units <= sms ? seg + 0.25 * states : std::max(seg, share + seg / 2) + 0.35 * states * units / sms) + start;
    };
    a.seg = ssm::kWhole;
    double best = 0.85 * cost(longest);
    for (int seg = ssm::kSegment; seg < longest; seg += ssm::kSegment)
        if (cost(seg) < best) best = cost(seg), a.seg = seg;
    const long long state = static_cast<long long>(a.H) * P * S, states = 2 * (a.T / (128 * ssm::kSegment));
    a.ws_states = states;
    a.ws = static_cast<float*>(workspace);
    a.ws_decay = a.ws + states * state;
    if (a.seg < ssm::kWhole) {
        const long long grid = a.T / 128 / a.seg * per_seg;
        e = ahead<P, S>(a, maps, static_cast<unsigned>(grid), stream);
        if (e != cudaSuccess) return e;
    }
    const long long grid = (a.T / 128 / a.seg + a.num_seqs) * per_seg;
    if (grid >= 1LL << 31) return cudaErrorInvalidConfiguration;
    return run<P, S>(a, maps, static_cast<unsigned>(grid), stream);
}

}  // namespace

void launch_ssm_steps(SsmArgs a, int S, cudaStream_t stream) {
    a.tiles = a.P / ssm::kRows;
    const unsigned grid = static_cast<unsigned>(a.num_seqs) * a.H * a.tiles;
    if (S == 64) {
        if (!a.cu) ssm::ssm_steps_kernel<64, 4, true><<<grid, ssm::kRows / 2 * 4, 0, stream>>>(a);
        else ssm::ssm_steps_kernel<64, 4, false><<<grid, ssm::kRows / 2 * 4, 0, stream>>>(a);
    } else {
        if (!a.cu) ssm::ssm_steps_kernel<128, 8, true><<<grid, ssm::kRows / 2 * 8, 0, stream>>>(a);
        else ssm::ssm_steps_kernel<128, 8, false><<<grid, ssm::kRows / 2 * 8, 0, stream>>>(a);
    }
}

// Two states for every segment that a call of T tokens can have, and their decays.
size_t ssm_workspace_bytes(int, long long T, int H, int P, int S) {
    return static_cast<size_t>(2 * (T / (128 * ssm::kSegment))) * H * (static_cast<size_t>(P) * S + 1) * sizeof(float);
}

cudaError_t launch_ssm_prefill(const SsmArgs& args, int S, long long max_len, void* workspace, cudaStream_t stream) {
    // Up to 16 tokens: a chunk's time does not depend on its tokens, a step's does.  64 heads of 64, N = 128, gated, us,
    // steps / chunks: 32 sequences of 12 tokens 80 / 109, of 16 101 / 109, of 20 125 / 109; 128 of 16 443 / 450; 1 of 16 21 / 19.
    if (max_len <= kSsmSteps) {
        launch_ssm_steps(args, S, stream);
        return cudaGetLastError();
    }
    SsmArgs a = args;
    if (a.polls == 0 || a.polls > ssm::kPolls) a.polls = ssm::kPolls;
    if (a.P == 64) return S == 64 ? chunks<64, 64>(a, max_len, workspace, stream) : chunks<64, 128>(a, max_len, workspace, stream);
    return S == 64 ? chunks<128, 64>(a, max_len, workspace, stream) : chunks<128, 128>(a, max_len, workspace, stream);
}

}  // namespace gdn
