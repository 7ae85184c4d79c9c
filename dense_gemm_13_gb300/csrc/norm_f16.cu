// norm_f16.cu -- the norm's kernels with an output in 16 or 32 bits, rows and residual in FP16.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm_f16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    return launch_norm_lay<false, GEMM_F16>(a, s, num_sms, st);
}

}  // namespace g13
