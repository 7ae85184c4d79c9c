// w4_capi.cpp -- the C entry points of 4-bit weights with group scales.
#include "w4.h"

#include <algorithm>
#include <cmath>
#include <cstring>

#include "device.h"
#include "dispatch.h"

using namespace g13;

namespace {

bool on(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool is16(int dtype) { return dtype == GEMM_F16 || dtype == GEMM_BF16; }

// Whether a weight of these sizes exists (INVALID_ARG) and is taken (UNSUPPORTED).
int check_weight(int64_t N, int64_t K, int64_t group) {
    if (N < 0 || K < 1 || group < 32 || group % 32 != 0) return GEMM_ERR_INVALID_ARG;
    // blocks of 512 bytes are counted in 32 bits
    if (N > kW4MaxN || K > kW4MaxK || group > kW4MaxK || w4_tiles(N) * w4_blocks(K) >= (int64_t(1) << 31))
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

int check_convert(int dtype, int scale_dtype, int64_t N, int64_t K, int64_t group, const void* matrix, int64_t ld,
                  const void* codes, const void* scales, const void* zeros) {
    if (dtype_size(dtype) == 0 || !is16(scale_dtype)) return GEMM_ERR_INVALID_ARG;
    const int rc = check_weight(N, K, group);
    if (rc != GEMM_OK) return rc;
    if (ld < K) return GEMM_ERR_INVALID_ARG;
    if (ld > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (N == 0) return GEMM_OK;
    if (!matrix || !codes || !scales) return GEMM_ERR_INVALID_ARG;
    if (!on(matrix, dtype_size(dtype)) || !on(codes, 16) || !on(scales, 16) || !on(zeros, 16))
        return GEMM_ERR_MISALIGNED;
    int sms = 0;
    return usable_device(&sms) ? GEMM_OK : GEMM_ERR_NO_DEVICE;
}

}  // namespace

extern "C" {

int64_t gemm_w4_codes_bytes(int64_t N, int64_t K) {
    return check_weight(N, K, 32) == GEMM_OK ? w4_tiles(N) * w4_blocks(K) * 512 : 0;
}
int64_t gemm_w4_scales_count(int64_t N, int64_t K, int64_t group) {
    return check_weight(N, K, group) == GEMM_OK ? w4_tiles(N) * 16 * w4_groups(K, group) : 0;
}

int gemm_w4_quantize(gemm_dtype_t dtype, gemm_dtype_t scale_dtype, int64_t N, int64_t K, int64_t group,
                     const void* src, int64_t ld, void* codes, void* scales, void* zeros, void* stream) {
    const int rc = check_convert(dtype, scale_dtype, N, K, group, src, ld, codes, scales, zeros);
    if (rc != GEMM_OK || N == 0) return rc;
    return cuda_status(launch_w4_quantize(dtype, scale_dtype, N, K, group, src, ld, static_cast<uint8_t*>(codes), scales,
                                          static_cast<uint8_t*>(zeros), static_cast<cudaStream_t>(stream)));
}

int gemm_w4_pack(int64_t N, int64_t K, int64_t group, const void* q, int64_t ldq, const void* s, int64_t lds,
                 const void* z, int64_t ldz, void* codes, void* scales, void* zeros, void* stream) {
    const int rc = check_weight(N, K, group);
    if (rc != GEMM_OK) return rc;
    const int64_t lim = int64_t(1) << 40, groups = w4_groups(K, group);
    if (ldq < K || lds < groups || (z && ldz < groups) || (z != nullptr) != (zeros != nullptr))
        return GEMM_ERR_INVALID_ARG;
    if (ldq > lim || lds > lim || ldz > lim) return GEMM_ERR_UNSUPPORTED;
    if (N == 0) return GEMM_OK;
    if (!q || !s || !codes || !scales) return GEMM_ERR_INVALID_ARG;
    if (!on(s, 2) || !on(codes, 16) || !on(scales, 16) || !on(zeros, 16)) return GEMM_ERR_MISALIGNED;
    int sms = 0;
    if (!usable_device(&sms)) return GEMM_ERR_NO_DEVICE;
    return cuda_status(launch_w4_pack(N, K, group, static_cast<const uint8_t*>(q), ldq, s, lds,
                                      static_cast<const uint8_t*>(z), ldz, static_cast<uint8_t*>(codes), scales,
                                      static_cast<uint8_t*>(zeros), static_cast<cudaStream_t>(stream)));
}

int gemm_w4_dequantize(gemm_dtype_t dtype, gemm_dtype_t scale_dtype, int64_t N, int64_t K, int64_t group,
                       const void* codes, const void* scales, const void* zeros, void* dst, int64_t ld, void* stream) {
    const int rc = check_convert(dtype, scale_dtype, N, K, group, dst, ld, codes, scales, zeros);
    if (rc != GEMM_OK || N == 0) return rc;
    return cuda_status(launch_w4_dequantize(dtype, scale_dtype, N, K, group, static_cast<const uint8_t*>(codes), scales,
                                            static_cast<const uint8_t*>(zeros), dst, ld,
                                            static_cast<cudaStream_t>(stream)));
}

int gemm_w4_run(const gemm_w4_desc_t* desc, const void* X, const void* codes, const void* scales, const void* zeros,
                void* Y, const void* bias, const void* residual, float alpha, void* stream) {
    if (!desc) return GEMM_ERR_INVALID_ARG;
    gemm_w4_desc_t d = *desc;
    if (dtype_size(d.dtype) == 0 || dtype_size(d.out_dtype) == 0) return GEMM_ERR_INVALID_ARG;
    if (d.act != GEMM_ACT_NONE && d.act != GEMM_ACT_GELU_ERF && d.act != GEMM_ACT_RELU)
        return d.act == GEMM_ACT_SOFTMAX ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_ARG;
    if ((d.has_zeros != 0 && d.has_zeros != 1) || (d.has_bias != 0 && d.has_bias != 1) ||
        (d.has_residual != 0 && d.has_residual != 1) || d.M < 0 || (d.flags & ~GEMM_FLAG_TEST_STALL))
        return GEMM_ERR_INVALID_ARG;
    const int rc = check_weight(d.N, d.K, d.group);
    if (rc != GEMM_OK) return rc;
    if (!is16(d.dtype) || d.M > kW4MaxTokens) return GEMM_ERR_UNSUPPORTED;
    if (d.ldx == 0) d.ldx = d.K;
    if (d.ldy == 0) d.ldy = std::max<int64_t>(d.N, 1);
    if (d.ldr == 0) d.ldr = d.ldy;
    if (d.ldx < d.K || d.ldy < d.N || d.ldr < d.N) return GEMM_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 40;
    if (d.ldx > lim || d.ldy > lim || d.ldr > lim) return GEMM_ERR_UNSUPPORTED;
    if ((d.has_bias != 0) != (bias != nullptr) || (d.has_residual != 0) != (residual != nullptr))
        return GEMM_ERR_INVALID_ARG;
    if (d.M == 0 || d.N == 0) return GEMM_OK;
    if (!X || !codes || !scales || !Y || (d.has_zeros != 0) != (zeros != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!on(X, 2) || !on(codes, 16) || !on(scales, 16) || !on(zeros, 16) || !on(Y, dtype_size(d.out_dtype)) ||
        !on(bias, 4) || !on(residual, 4))
        return GEMM_ERR_MISALIGNED;
    int sms = 0;
    if (!usable_device(&sms)) return GEMM_ERR_NO_DEVICE;
    W4Args a{};
    a.dtype = d.dtype;
    a.M = d.M;
    a.N = d.N;
    a.K = d.K;
    a.group = d.group;
    a.ldx = d.ldx;
    a.x = X;
    a.codes = static_cast<const uint8_t*>(codes);
    a.scales = scales;
    a.zeros = static_cast<const uint8_t*>(zeros);
    a.e.C = Y;
    a.e.ldc = d.ldy;
    a.e.bias = static_cast<const float*>(bias);
    a.e.R = static_cast<const float*>(residual);
    a.e.ldr = d.ldr;
    a.e.M = d.M;
    a.e.N = d.N;
    a.e.alpha = alpha;
    a.e.beta = d.beta;
    a.e.out_dtype = d.out_dtype;
    a.e.act = d.act;
    a.timeout_ns = (d.timeout_ms ? d.timeout_ms : 2000u) * uint64_t(1000000);
    a.flags = d.flags;
    // four neighbouring columns as one access
    const int64_t size = dtype_size(d.out_dtype);
    a.e.c_vec = on(Y, 4 * size) && (d.M <= 1 || d.ldy % 4 == 0);
    a.e.r_vec = on(residual, 16) && (d.M <= 1 || d.ldr % 4 == 0);
    if (const int splits = w4_tc_splits(a, sms)) return cuda_status(launch_w4_tc(a, splits, static_cast<cudaStream_t>(stream)));
    return cuda_status(launch_w4(w4_choose(d.M, d.N, d.K, d.group, sms), a, sms, static_cast<cudaStream_t>(stream)));
}

void gemm_w4_desc_init(gemm_w4_desc_t* d) {
    if (!d) return;
    std::memset(d, 0, sizeof(*d));
    d->dtype = d->out_dtype = GEMM_BF16;
    d->group = 128;
    d->act = GEMM_ACT_NONE;
    d->beta = 1.0f;
}

}  // extern "C"
