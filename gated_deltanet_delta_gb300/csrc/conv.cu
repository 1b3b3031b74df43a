// conv.cu -- launch of the short convolution (conv.cuh).
#include <atomic>

#include "conv.cuh"
#include "host.h"
#include "launch.h"

namespace gdn {
namespace {

template <int TAPS, bool F16>
cudaError_t run(const ConvArgs& a, cudaStream_t stream) {
    const unsigned blocks = (a.C / 8 + conv::kThreads - 1) / conv::kThreads;
    if (!a.cu) {
        conv::short_conv_step_kernel<TAPS, F16><<<dim3(a.num_seqs, blocks), conv::kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long tiles = (a.T + conv::kTile - 1) / conv::kTile;
    // A CTA of the ring takes 28 us for its 128 tokens and four are on an SM: with fewer than two per SM the kernel of 32 tokens is done
    // sooner (8192 channels, us, that one / the ring: 0.8 CTAs per SM 21 / 28, 1.7: 35 / 36, 2.5: 49 / 45, 5.1: 85 / 84, 10: 154 / 141).
    if (tiles * blocks >= 2 * sms) {
        static std::atomic<unsigned long long> done{0};
        e = raise_smem(conv::short_conv_ring_kernel<TAPS, F16>, conv::kRing, done);
        if (e != cudaSuccess) return e;
        conv::short_conv_ring_kernel<TAPS, F16><<<dim3(static_cast<unsigned>(tiles), blocks), conv::kThreads, conv::kRing, stream>>>(a);
    } else {
        const dim3 grid(static_cast<unsigned>((a.T + conv::kTokens - 1) / conv::kTokens), blocks);
        conv::short_conv_kernel<TAPS, F16><<<grid, conv::kThreads, 0, stream>>>(a);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv::short_conv_history_kernel<TAPS, F16><<<dim3(a.num_seqs, blocks), conv::kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <int TAPS>
cudaError_t run_taps(const ConvArgs& a, bool f16, cudaStream_t stream) {
    return f16 ? run<TAPS, true>(a, stream) : run<TAPS, false>(a, stream);
}

}  // namespace

cudaError_t launch_conv(ConvArgs a, int taps, bool f16, cudaStream_t stream) {
    if (a.polls == 0 || a.polls > conv::kWaitPolls) a.polls = conv::kWaitPolls;
    if (taps == 2) return run_taps<2>(a, f16, stream);
    if (taps == 3) return run_taps<3>(a, f16, stream);
    return run_taps<4>(a, f16, stream);
}

}  // namespace gdn
