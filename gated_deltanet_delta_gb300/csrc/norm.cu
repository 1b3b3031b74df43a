// norm.cu -- launch of the norm (norm.cuh).
#include "launch.h"
#include "norm.cuh"

namespace gdn {
namespace {

template <bool F16, bool F8, int R>
void run(const NormArgs& a, cudaStream_t stream) {
    const int pieces = a.C / 8;
    const int threads = ((pieces + R - 1) / R + 31) / 32 * 32, rows = threads >= 128 ? 1 : 128 / threads;
    norm::add_rms_norm_kernel<F16, F8, R><<<static_cast<unsigned>((a.T + rows - 1) / rows), dim3(threads, rows), 0, stream>>>(a);
}
template <bool F16, bool F8>
void run_r(const NormArgs& a, cudaStream_t stream) {
    const int pieces = a.C / 8;
    if (pieces <= 256) run<F16, F8, 1>(a, stream);
    else if (pieces <= 1024) run<F16, F8, 2>(a, stream);
    else if (pieces <= 2048) run<F16, F8, 4>(a, stream);
    else run<F16, F8, 8>(a, stream);
}

}  // namespace

void launch_norm(const NormArgs& a, bool f16, bool f8, cudaStream_t stream) {
    if (f8) f16 ? run_r<true, true>(a, stream) : run_r<false, true>(a, stream);
    else f16 ? run_r<true, false>(a, stream) : run_r<false, false>(a, stream);
}

}  // namespace gdn
