// conv.cu -- launch of the short convolution (conv.cuh).
#include "conv.cuh"
#include "launch.h"

namespace gdn {
namespace {

template <int TAPS, bool F16>
void run(const ConvArgs& a, cudaStream_t stream) {
    const unsigned blocks = (a.C / 8 + conv::kThreads - 1) / conv::kThreads;
    if (!a.cu) {
        conv::short_conv_step_kernel<TAPS, F16><<<dim3(a.num_seqs, blocks), conv::kThreads, 0, stream>>>(a);
        return;
    }
    const dim3 grid(static_cast<unsigned>((a.T + conv::kTokens - 1) / conv::kTokens), blocks);
    conv::short_conv_kernel<TAPS, F16><<<grid, conv::kThreads, 0, stream>>>(a);
    conv::short_conv_history_kernel<TAPS, F16><<<dim3(a.num_seqs, blocks), conv::kThreads, 0, stream>>>(a);
}
template <int TAPS>
void run_taps(const ConvArgs& a, bool f16, cudaStream_t stream) {
    f16 ? run<TAPS, true>(a, stream) : run<TAPS, false>(a, stream);
}

}  // namespace

void launch_conv(const ConvArgs& a, int taps, bool f16, cudaStream_t stream) {
    if (taps == 2) run_taps<2>(a, f16, stream);
    else if (taps == 3) run_taps<3>(a, f16, stream);
    else run_taps<4>(a, f16, stream);
}

}  // namespace gdn
