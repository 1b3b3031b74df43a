// attn.cu -- launch of attention over a paged cache: choice of the kernel and of its grid.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "attn_rows.cuh"
#include "attn_tiles.cuh"
#include "host.h"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kMaxCtas = 608;      // of the row kernel; the workspace has two partial slots for each
constexpr int kMaxTileCtas = 160;  // of the tile kernel, likewise
constexpr size_t kJoinBytes = kMaxCtas * sizeof(AttnJoin);  // at the workspace's start
static_assert(kJoinBytes % 16 == 0, "the partials are read by 16 bytes");

// Raises a kernel's shared-memory limit once per device.
template <typename K>
cudaError_t raise_smem(K kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

// A cache as rows of D elements, in boxes of `box` rows and `line` bytes (a row, or 128 bytes of it), with the
// swizzle of that width, or none.
bool encode_cache(CUtensorMap* map, const void* base, long long rows, int D, int box, int line, bool swizzle, bool f8, bool f16) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const int size = f8 ? 1 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * size};
    const cuuint32_t shape[2] = {static_cast<cuuint32_t>(line / size), static_cast<cuuint32_t>(box)};
    const cuuint32_t step[2] = {1, 1};
    const CUtensorMapDataType type = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : (f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
    const CUtensorMapSwizzle sw = !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : (line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    return fn(map, type, 2, const_cast<void*>(base), dims, strides, shape, step, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Chooses a.box, the rows of a box: a power of two up to `most` that divides a page; 0 (no TMA) where that is
// below `least`, or where a row's number passes the coordinates' 32 bits.  Makes the maps.
cudaError_t make_maps(AttnArgs& a, AttnMaps& maps, int D, bool f8, int least, int most, int line, bool swizzle) {
    std::memset(&maps, 0, sizeof(maps));
    const long long rows = a.num_pages * a.Hkv * a.page_size;
    a.box = std::min(a.page_size & -a.page_size, most);
    if (a.box < least || rows < a.box || rows >= 1LL << 31) a.box = 0;
    if (a.box == 0) return cudaSuccess;
    return encode_cache(&maps.k, a.kc, rows, D, a.box, line, swizzle, f8, a.f16) &&
                   encode_cache(&maps.v, a.vc, rows, D, a.box, line, swizzle, f8, a.f16)
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// The joining kernel starts while the main kernel still runs (programmatic dependent launch) and waits
// for it before it reads the partials.
template <int D>
cudaError_t launch_combine(const AttnArgs& a, int R, int grid, cudaStream_t stream) {
    const int RB = std::min(R, attn::kCombineThreads / (D / 4));  // a row per group of threads
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, (R + RB - 1) / RB);
    cfg.blockDim = dim3(attn::kCombineThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn::attn_combine_kernel<D>, a, R, RB);
}

template <int D, bool F16, bool F8>
cudaError_t launch_rows(AttnArgs a, cudaStream_t stream) {
    using C = attn::RowsCfg<D, F8>;
    static std::atomic<unsigned long long> done{0};
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = raise_smem(attn::attn_rows_kernel<D, F16, F8>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    a.tq = std::max(1, attn::kRowsTile / a.G);
    a.ov = 1;
    a.min_per = 3;
    AttnMaps maps;
    // the scales of a box come by copies that begin on 16-byte boundaries
    const bool tma = F8 && (reinterpret_cast<uintptr_t>(a.ks) | reinterpret_cast<uintptr_t>(a.vs)) % 16 == 0;
    if (tma) {
        e = make_maps(a, maps, D, F8, 16, C::TK, C::LINE, true);
        if (e != cudaSuccess) return e;
    } else {
        std::memset(&maps, 0, sizeof(maps));
        a.box = 0;
    }
    const int grid = std::min(sms * C::OCC, kMaxCtas);
    attn::attn_rows_kernel<D, F16, F8><<<grid, attn::kRowsNT, C::SMEM, stream>>>(a, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_combine<D>(a, attn::kRowsTile, grid, stream);
}

template <int D, bool F16, bool F8>
cudaError_t launch_tiles(AttnArgs a, cudaStream_t stream) {
    using C = attn::TilesCfg<D, F8>;
    static std::atomic<unsigned long long> done{0};
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = raise_smem(attn::attn_tiles_kernel<D, F16, F8>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    // the split of registers among roles waits forever where the launch has fewer than it adds up to
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, attn::attn_tiles_kernel<D, F16, F8>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < attn::kRegsLaunch) return cudaErrorInvalidConfiguration;
    a.tq = C::R / a.G;
    a.ov = 6;
    a.min_per = 8;
    // boxes of at least 8 rows, the swizzle's period; 8 bits: whole rows, unswizzled, into the staging ring
    AttnMaps maps;
    e = make_maps(a, maps, D, F8, 8, C::BOX, F8 ? D : 128, !F8);
    if (e != cudaSuccess) return e;
    const int grid = std::min(sms, kMaxTileCtas);
    attn::attn_tiles_kernel<D, F16, F8><<<grid, attn::kTilesNT, C::SMEM, stream>>>(a, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_combine<D>(a, C::R, grid, stream);
}

template <int D, bool F16, bool F8>
cudaError_t launch_any(const AttnArgs& a, int max_q, cudaStream_t stream) {
    // The row kernel reads a key once per 16 rows that share it, the tile kernel once.  Measured with 32 sequences of up
    // to 8192 keys, 1024 values each, and 8 heads per key head, row kernel and tile kernel.  16 bits: heads of 128, 16 rows
    // 106 and 117 us, 24 rows 172 and 117 us; heads of 256, 16 rows 116 and 109 us, 32 rows 217 and 113 us (2 rows,
    // 64 sequences, 199 and 189 us: the rule leaves aside that this width is always the tile kernel's).  8 bits, where the tile kernel has to widen every key
    // tile first: heads of 128, 32 rows 119 and 215 us, 64 rows 221 and 225 us, 128 rows 292 and 239 us; heads of
    // 64, 64 rows 287 and 333 us, 128 rows 379 and 383 us; heads of 256, 16 rows 84 and 115 us, 32 rows 151 and 116 us.
    const int most = F8 && D <= 128 ? 4 * attn::kRowsTile : attn::kRowsTile;
    return static_cast<long long>(std::max(max_q, 1)) * a.G <= most && a.G <= attn::kRowsTile
               ? launch_rows<D, F16, F8>(a, stream)
               : launch_tiles<D, F16, F8>(a, stream);
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, bool f8, int max_q, cudaStream_t stream) {
    if (a.f16) return f8 ? launch_any<D, true, true>(a, max_q, stream) : launch_any<D, true, false>(a, max_q, stream);
    return f8 ? launch_any<D, false, true>(a, max_q, stream) : launch_any<D, false, false>(a, max_q, stream);
}
}  // namespace

size_t attn_workspace_bytes(int D) {
    const size_t rows = static_cast<size_t>(kMaxCtas) * attn::kRowsTile;
    const size_t tiles = static_cast<size_t>(kMaxTileCtas) * (D == 256 ? attn::TilesCfg<256, false>::R : attn::TilesCfg<128, false>::R);
    return kJoinBytes + std::max(rows, tiles) * 2 * (D + 2) * sizeof(float);
}

cudaError_t launch_attn(const AttnArgs& args, void* workspace, int D, bool f8, int max_q, cudaStream_t stream) {
    AttnArgs a = args;
    if (a.polls == 0 || a.polls > attn::kWaitPolls) a.polls = attn::kWaitPolls;
    a.joins = static_cast<AttnJoin*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kJoinBytes);
    if (D == 64) return launch_d<64>(a, f8, max_q, stream);
    if (D == 128) return launch_d<128>(a, f8, max_q, stream);
    return launch_d<256>(a, f8, max_q, stream);
}

}  // namespace gdn
