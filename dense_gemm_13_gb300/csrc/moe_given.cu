// moe_given.cu -- the mixture-of-experts layer on a choice made beforehand.
#include "moe_kernel.cuh"

namespace g13 {

cudaError_t launch_moe_given(const MoeArgs& a, int grid, cudaStream_t st) { return launch_moe_kernels<true>(a, grid, st); }

}  // namespace g13
