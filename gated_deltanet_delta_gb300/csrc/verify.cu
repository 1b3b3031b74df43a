// verify.cu -- launch of the draft verification (verify.cuh).
#include "host.h"
#include "launch.h"
#include "verify.cuh"

namespace gdn {

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
    const int chunks = (a.V + verify::kChunk - 1) / verify::kChunk;
    // Four CTAs fit an SM.  Eight per sequence while they all run at once (64 sequences of 131072: 16.8 us,
    // with four 17.3); beyond that four (255 sequences of 100003: 44.4 us, with eight 48.9, with two 44.5).
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    int C = static_cast<long long>(a.N) * 8 <= static_cast<long long>(sms) * 4 ? 8 : 4;
    // a CTA has 8 warps: no more CTAs than the row has chunks for
    while (C > 1 && chunks < C * 8) C /= 2;
    const int per = (chunks + C - 1) / C + 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * C);
    cfg.blockDim = dim3(verify::kThreads);
    cfg.dynamicSmemBytes = per * sizeof(unsigned long long);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify::draft_verify_kernel, a);
}

}  // namespace gdn
