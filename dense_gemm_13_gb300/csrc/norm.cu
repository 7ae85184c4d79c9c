// norm.cu -- the norm's kernels with an output in 16 or 32 bits and rows and residual of any types, and the choice
// between all of them.
#include "norm_kernel.cuh"

namespace g13 {

cudaError_t launch_norm_any(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    return launch_norm_lay<false, ANY>(a, s, num_sms, st);
}

namespace {

struct Rows {
    const void* p;
    int type;
    int64_t ld;
    int unit() const { return type == GEMM_F32 ? 4 : 8; }  // elements of 16 bytes
    int first() const { return static_cast<int>(reinterpret_cast<uintptr_t>(p) / (16 / unit()) & 7); }
    int step() const { return static_cast<int>(ld & 7); }
};

// The rows' lay, and with it s.phase and s.phase_step.
NormLay lay_of(const NormArgs& a, bool f8, NormShape& s) {
    const gemm_norm_desc_t& d = a.d;
    const Rows all[4] = {{a.x, d.dtype, d.ldx}, {a.r, d.residual_dtype, d.ldr}, {a.h, d.residual_dtype, d.ldh},
                         {f8 ? nullptr : a.y, d.out_dtype, d.ldy}};
    const bool weight = reinterpret_cast<uintptr_t>(a.w) % 16 == 0, many = d.rows > 1;
    s.wide_weight = weight && d.weight_dtype != GEMM_F32;
    int unit = 0;  // of a 16-bit array, if there is one
    for (const Rows& r : all) {
        if (!r.p || r.unit() <= unit) continue;
        unit = r.unit();
        s.phase = r.first() & (unit - 1);
        s.phase_step = many ? r.step() & (unit - 1) : 0;
    }
    bool aligned = weight, phased = s.cols <= norm_phased(f8) && (weight || !f8);
    for (const Rows& r : all) {
        if (!r.p) continue;
        const int mask = r.unit() - 1;
        aligned = aligned && (r.first() & mask) == 0 && (!many || (r.step() & mask) == 0);
        phased = phased && ((r.first() ^ s.phase) & mask) == 0 && (!many || ((r.step() ^ s.phase_step) & mask) == 0);
    }
    return aligned ? ALIGNED : phased ? PHASED : SINGLES;
}

}  // namespace

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
    s.lay = lay_of(a, f8, s);
    // (d.residual_dtype is x's where there is no residual)
    const int type = d.dtype == d.residual_dtype ? static_cast<int>(d.dtype) : ANY;
    if (type == GEMM_BF16) return f8 ? launch_norm8_bf16(a, s, num_sms, st) : launch_norm_bf16(a, s, num_sms, st);
    if (type == GEMM_F16) return f8 ? launch_norm8_f16(a, s, num_sms, st) : launch_norm_f16(a, s, num_sms, st);
    return f8 ? launch_norm8_any(a, s, num_sms, st) : launch_norm_any(a, s, num_sms, st);
}

}  // namespace g13
