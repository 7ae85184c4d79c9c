// norm.cu -- the norm's kernels with an output in 16 or 32 bits, and the choice between the two kinds.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm8(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st) {
    const gemm_norm_desc_t& d = a.d;
    const bool f8 = a.scales != nullptr;
    NormShape s{};
    s.cols = static_cast<int>(d.cols);
    s.inv.hi = static_cast<float>(1.0 / static_cast<double>(d.cols));
    s.inv.lo = static_cast<float>(1.0 / static_cast<double>(d.cols) - s.inv.hi);
    s.rows = d.rows;
    s.rows_all = f8 ? fp4_row_tiles(d.rows) * 128 : d.rows;
    s.row_bytes = fp4_row_bytes(kMxfp8, d.cols);
    s.col_tiles = fp4_col_tiles(kMxfp8, d.cols);
    return f8 ? launch_norm8(a, s, num_sms, st) : launch_norm_kind<false>(a, s, num_sms, st);
}

}  // namespace g13
