// cache.cu -- launch of the cache write and read kernels (cache.cuh).
#include "cache.cuh"
#include "launch.h"

namespace gdn {
namespace {

// 64 tokens per CTA keep four rows of 128 in flight per group; with few tokens there are not enough
// CTAs that way, and 16 tokens each take more of them.  Measured with 8 heads of 128, 8 bits, 64 and 16 tokens per
// CTA: write, 1024 tokens 3.5 and 3.0 us, 4096 tokens 6.9 and 7.4 us, 16384 tokens 21.3 and 25.8 us; read, 1024
// tokens 3.2 and 3.1 us, 4096 tokens 4.8 and 6.3 us, 16384 tokens 13.6 and 21.7 us.
template <int D, bool F16, bool F8>
void write(const CacheMoveArgs& a, cudaStream_t stream) {
    if (a.T >= 2048) {
        const dim3 grid(static_cast<unsigned>((a.T + 63) / 64), a.H, 2);
        cache::attn_cache_write_kernel<D, F16, F8, 64><<<grid, cache::kThreads, 0, stream>>>(a);
    } else {
        const dim3 grid(static_cast<unsigned>((a.T + 15) / 16), a.H, 2);
        cache::attn_cache_write_kernel<D, F16, F8, 16><<<grid, cache::kThreads, 0, stream>>>(a);
    }
}
template <int D, bool F16, bool F8>
void read(const CacheMoveArgs& a, cudaStream_t stream) {
    if (a.T >= 2048) {
        const dim3 grid(static_cast<unsigned>((a.T + 63) / 64), a.H, 2);
        cache::attn_cache_read_kernel<D, F16, F8, 64><<<grid, cache::kThreads, 0, stream>>>(a);
    } else {
        const dim3 grid(static_cast<unsigned>((a.T + 15) / 16), a.H, 2);
        cache::attn_cache_read_kernel<D, F16, F8, 16><<<grid, cache::kThreads, 0, stream>>>(a);
    }
}
template <int D>
void write_d(const CacheMoveArgs& a, bool f16, bool f8, cudaStream_t stream) {
    // an unquantised write moves 16-bit words whatever they mean
    if (!f8) write<D, false, false>(a, stream);
    else if (f16) write<D, true, true>(a, stream);
    else write<D, false, true>(a, stream);
}
template <int D>
void read_d(const CacheMoveArgs& a, bool f16, bool f8, cudaStream_t stream) {
    if (!f8) read<D, false, false>(a, stream);
    else if (f16) read<D, true, true>(a, stream);
    else read<D, false, true>(a, stream);
}
}  // namespace

void launch_cache_write(const CacheMoveArgs& a, int D, bool f16, bool f8, cudaStream_t stream) {
    if (D == 64) write_d<64>(a, f16, f8, stream);
    else if (D == 128) write_d<128>(a, f16, f8, stream);
    else write_d<256>(a, f16, f8, stream);
}
void launch_cache_read(const CacheMoveArgs& a, int D, bool f16, bool f8, cudaStream_t stream) {
    if (D == 64) read_d<64>(a, f16, f8, stream);
    else if (D == 128) read_d<128>(a, f16, f8, stream);
    else read_d<256>(a, f16, f8, stream);
}

}  // namespace gdn
