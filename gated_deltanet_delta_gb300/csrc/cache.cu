// cache.cu -- launch of the cache write and read kernels (cache.cuh).
#include "cache.cuh"
#include "launch.h"

namespace gdn {
namespace {

// 64 tokens per CTA keep four rows of 128 in flight per group; with few tokens there are not enough
// CTAs that way, and 16 tokens each take more of them.  Measured with 8 heads of 128, 8 bits, memory that L2 does not
// hold, 64 and 16 tokens per CTA: write, 1024 tokens 3.8 and 3.1 us, 2048 tokens 5.4 and 5.4 us, 4096 tokens 7.8 and
// 8.6 us, 16384 tokens 20.4 and 26.1 us; read, 256 tokens 2.6 and 2.4 us, 1024 tokens 3.5 and 3.7 us, 4096 tokens
// 6.5 and 8.1 us, 16384 tokens 18.6 and 26.0 us.
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
