// norm8_f16.cu -- the norm's kernels with an output in mxfp8, rows and residual in FP16.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm8_f16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    return launch_norm_lay<true, GEMM_F16>(a, s, num_sms, st);
}

}  // namespace g13
