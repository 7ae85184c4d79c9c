// norm8.cu -- the norm's kernels with an output in mxfp8, rows and residual of any types.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm8_any(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    return launch_norm_lay<true, ANY>(a, s, num_sms, st);
}

}  // namespace g13
