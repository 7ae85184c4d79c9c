// norm_bf16.cu -- the norm's kernels with an output in 16 or 32 bits, rows and residual in BF16.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm_bf16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    return launch_norm_lay<false, GEMM_BF16>(a, s, num_sms, st);
}

}  // namespace g13
