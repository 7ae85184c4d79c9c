// norm_capi.cpp -- the C entry point of the root-mean-square norm.
#include "norm.h"

#include <cmath>
#include <cstring>

#include "device.h"
#include "dispatch.h"
#include "fp4.cuh"
#include "internal.h"

using namespace g13;

namespace {

bool on(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check(gemm_norm_desc_t& d) {
    if (dtype_size(d.dtype) == 0 || dtype_size(d.residual_dtype) == 0 || dtype_size(d.weight_dtype) == 0 ||
        dtype_size(d.out_dtype) == 0)
        return GEMM_ERR_INVALID_ARG;
    if ((d.has_residual != 0 && d.has_residual != 1) || (d.mxfp8 != 0 && d.mxfp8 != 1)) return GEMM_ERR_INVALID_ARG;
    if (d.rows < 0 || d.cols < 1 || !(d.eps >= 0.0f) || !std::isfinite(d.eps) || !std::isfinite(d.weight_offset))
        return GEMM_ERR_INVALID_ARG;
    if (!d.has_residual) d.residual_dtype = d.dtype;
    if (d.residual_dtype != d.dtype && d.residual_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    for (int64_t* ld : {&d.ldx, &d.ldr, &d.ldh, &d.ldy}) {
        if (*ld == 0) *ld = d.cols;
        if (*ld < d.cols) return GEMM_ERR_INVALID_ARG;
        if (*ld > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    }
    // (the kernels' offsets stay in 64 bits, the scales' tiles as in gemm_fp8_quantize)
    if (d.cols > kNormMaxCols || d.rows > (int64_t(1) << 31) - 256) return GEMM_ERR_UNSUPPORTED;
    if (d.mxfp8 && ((d.rows + 127) / 128 * 4) * ((d.cols + 255) / 256) >= (int64_t(1) << 30))
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

extern "C" {

void gemm_norm_desc_init(gemm_norm_desc_t* d) {
    if (!d) return;
    std::memset(d, 0, sizeof(*d));
    d->dtype = d->residual_dtype = d->weight_dtype = d->out_dtype = GEMM_BF16;
    d->eps = 1e-6f;
}

int gemm_rms_norm(const gemm_norm_desc_t* desc, const void* X, const void* residual, const void* weight, void* H,
                  void* Y, void* scales, void* stream) {
    if (!desc) return GEMM_ERR_INVALID_ARG;
    NormArgs a{};
    a.d = *desc;
    const int rc = check(a.d);
    if (rc != GEMM_OK) return rc;
    const gemm_norm_desc_t& d = a.d;
    if ((scales != nullptr) != (d.mxfp8 != 0) && d.rows > 0) return GEMM_ERR_INVALID_ARG;
    if (!d.has_residual && (residual || H)) return GEMM_ERR_INVALID_ARG;
    if (d.rows == 0) return GEMM_OK;
    if (!X || !Y || (d.has_residual && !residual)) return GEMM_ERR_INVALID_ARG;
    if (H && H == Y) return GEMM_ERR_INVALID_ARG;
    // in place: each element is read by the thread that writes it, at the same offset only
    const auto in_place = [&](const void* out, int type, int64_t ld, const void* in, int in_type, int64_t in_ld) {
        return out != in || (type == in_type && (ld == in_ld || d.rows == 1));
    };
    if (H && (!in_place(H, d.residual_dtype, d.ldh, X, d.dtype, d.ldx) ||
              !in_place(H, d.residual_dtype, d.ldh, residual, d.residual_dtype, d.ldr)))
        return GEMM_ERR_INVALID_ARG;
    if (d.mxfp8) {
        if (Y == X || Y == residual || Y == scales || scales == X || scales == residual || scales == H)
            return GEMM_ERR_INVALID_ARG;
    } else if (!in_place(Y, d.out_dtype, d.ldy, X, d.dtype, d.ldx) ||
               (residual && !in_place(Y, d.out_dtype, d.ldy, residual, d.residual_dtype, d.ldr))) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (weight && (weight == Y || weight == H || weight == scales)) return GEMM_ERR_INVALID_ARG;
    if (!on(X, dtype_size(d.dtype)) || !on(residual, dtype_size(d.residual_dtype)) ||
        !on(H, dtype_size(d.residual_dtype)) || !on(weight, dtype_size(d.weight_dtype)) ||
        !on(Y, d.mxfp8 ? 16 : dtype_size(d.out_dtype)) || !on(scales, 16))
        return GEMM_ERR_MISALIGNED;
    int sms = 0;
    if (!usable_device(&sms)) return GEMM_ERR_NO_DEVICE;
    a.x = X;
    a.r = residual;
    a.w = weight;
    a.h = H;
    a.y = Y;
    a.scales = static_cast<uint8_t*>(scales);
    return cuda_status(launch_rms_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
