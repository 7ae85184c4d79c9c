// fp4_capi.cpp -- the C entry points of the microscaled formats (gemm_fp4_*, gemm_fp8_*).
#include <algorithm>
#include <cstring>
#include <mutex>
#include <new>
#include <unordered_set>

#include "device.h"
#include "dispatch.h"
#include "fp4.cuh"
#include "fp4_gemm.h"

using namespace g13;

namespace {
struct BlockPlan {
    Problem p{};
    int format = 0;
    Fp4Config cfg{};
    int device = 0;
    int num_sms = 0;
    unsigned* d_status = nullptr;
};
}  // namespace
struct gemm_fp4_plan_s : BlockPlan {};
struct gemm_fp8_plan_s : BlockPlan {};

namespace {

std::mutex g_live_mu;
std::unordered_set<const void*> g_live4, g_live8;
std::unordered_set<const void*>& live(const gemm_fp4_plan_s*) { return g_live4; }
std::unordered_set<const void*>& live(const gemm_fp8_plan_s*) { return g_live8; }

template <typename P>
bool alive(const P* p) {
    if (!p) return false;
    std::lock_guard<std::mutex> lk(g_live_mu);
    return live(p).count(p) != 0;
}

bool format4(int f) { return f == GEMM_MXFP4 || f == GEMM_NVFP4; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Sizes that the kernels' grids and 32-bit TMA coordinates hold.
bool sizes_ok(int64_t rows, int64_t cols) {
    const int64_t lim = (int64_t(1) << 31) - 256;
    if (rows > lim || cols > lim) return false;
    return rows == 0 || cols == 0 || ((rows + 127) / 128 * 4) * ((cols + 255) / 256) < (int64_t(1) << 30);
}
int64_t scales_bytes(int format, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || !sizes_ok(rows, cols)) return 0;
    return fp4_row_tiles(rows) * fp4_col_tiles(format, cols) * kFp4TileBytes;
}

bool product_sizes_ok(int64_t M, int64_t N, int64_t K) {
    if (!sizes_ok(M, K) || !sizes_ok(N, K)) return false;
    // tile counts, and byte offsets along a row of C, are 32-bit in the kernel
    return N < (int64_t(1) << 30) &&
           (M == 0 || N == 0 || ((M + 127) / 128) * ((N + 127) / 128) < (int64_t(1) << 27));
}

int check_convert(int format, int dtype, int64_t rows, int64_t cols, int64_t ld, const void* matrix,
                  const float* tensor_scale, const void* codes, const void* scales) {
    if (dtype_size(dtype) == 0) return GEMM_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || ld < std::max<int64_t>(cols, 1)) return GEMM_ERR_INVALID_ARG;
    if (format != GEMM_NVFP4 && tensor_scale) return GEMM_ERR_INVALID_ARG;
    if (!sizes_ok(rows, cols)) return GEMM_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!matrix || !codes || !scales) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales)) return GEMM_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(matrix) % dtype_size(dtype) != 0 ||
        reinterpret_cast<uintptr_t>(tensor_scale) % 4 != 0)
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

int quantize(int format, int dtype, int64_t rows, int64_t cols, const void* src, int64_t ld,
             const float* tensor_scale, void* codes, void* scales, void* stream) {
    const int rc = check_convert(format, dtype, rows, cols, ld, src, tensor_scale, codes, scales);
    if (rc != GEMM_OK || rows == 0 || cols == 0) return rc;
    return cuda_status(launch_fp4_quantize(format, dtype, src, rows, cols, ld, tensor_scale,
                                           static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                           static_cast<cudaStream_t>(stream)));
}

int dequantize(int format, int dtype, int64_t rows, int64_t cols, const void* codes, const void* scales,
               const float* tensor_scale, void* dst, int64_t ld, void* stream) {
    const int rc = check_convert(format, dtype, rows, cols, ld, dst, tensor_scale, codes, scales);
    if (rc != GEMM_OK || rows == 0 || cols == 0) return rc;
    return cuda_status(launch_fp4_dequantize(format, dtype, static_cast<const uint8_t*>(codes),
                                             static_cast<const uint8_t*>(scales), tensor_scale, dst, rows,
                                             cols, ld, static_cast<cudaStream_t>(stream)));
}

int select_config(int format, int64_t M, int64_t N, int64_t K, int32_t num_sms, gemm_config_t* out) {
    if (!out || M < 0 || N < 0 || K < 0 || num_sms < 1) return GEMM_ERR_INVALID_ARG;
    if (!product_sizes_ok(M, N, K)) return GEMM_ERR_UNSUPPORTED;
    const Fp4Config c = fp4_choose(format, M, N, K, num_sms);
    std::memset(out, 0, sizeof(*out));
    out->kernel = GEMM_KERNEL_TC;
    out->bm = c.bn == 256 ? 256 : 128;
    out->variant = c.bn == 256 ? TC_VARIANT_PAIR : 0;
    out->bn = c.bn;
    out->bk = fp4_stage_k(format);
    out->split_k = c.splits;
    return GEMM_OK;
}

template <typename P>
int make_plan(int format, int64_t M, int64_t N, int64_t K, int64_t ldc, const gemm_epilogue_t* epilogue,
              P** out_plan) {
    gemm_epilogue_t e;
    gemm_epilogue_init(&e);
    e.b_layout = GEMM_B_NK;
    if (epilogue) e = *epilogue;
    e.stride_a = e.stride_b = e.stride_c = e.stride_r = 0;
    if (e.batch == 0) e.batch = 1;
    if (e.batch < 0) return GEMM_ERR_INVALID_ARG;
    if (e.batch > 1) return GEMM_ERR_UNSUPPORTED;
    Problem p;
    const int rc = make_problem(GEMM_BF16, M, N, K, std::max<int64_t>(K, 1),
                                std::max<int64_t>(e.b_layout == GEMM_B_KN ? N : K, 1), ldc, &e, &p);
    if (rc != GEMM_OK) return rc;
    if (p.epi.b_layout != GEMM_B_NK || p.epi.act == GEMM_ACT_SOFTMAX) return GEMM_ERR_UNSUPPORTED;
    if (!product_sizes_ok(M, N, K)) return GEMM_ERR_UNSUPPORTED;

    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 ||
        minor != 3)
        return GEMM_ERR_NO_DEVICE;
    P* pl = new (std::nothrow) P();
    if (!pl) return GEMM_ERR_OUT_OF_MEMORY;
    pl->p = p;
    pl->format = format;
    pl->device = dev;
    pl->num_sms = sms;
    pl->cfg = fp4_choose(format, M, N, K, sms);
    cudaError_t ce = cudaMalloc(reinterpret_cast<void**>(&pl->d_status), sizeof(unsigned));
    if (ce == cudaSuccess) ce = cudaMemset(pl->d_status, 0, sizeof(unsigned));
    if (ce != cudaSuccess) {
        if (pl->d_status) cudaFree(pl->d_status);
        delete pl;
        return cuda_status(ce);
    }
    try {
        std::lock_guard<std::mutex> lk(g_live_mu);
        live(pl).insert(pl);
    } catch (...) {
        cudaFree(pl->d_status);
        delete pl;
        return GEMM_ERR_OUT_OF_MEMORY;
    }
    *out_plan = pl;
    return GEMM_OK;
}

int run(const BlockPlan* plan, const void* a_codes, const void* a_scales, const float* a_tensor_scale,
        const void* b_codes, const void* b_scales, const float* b_tensor_scale, void* C, const void* bias,
        const void* residual, float alpha, void* stream) {
    const Problem& p = plan->p;
    const gemm_epilogue_t& ep = p.epi;
    if (plan->format != GEMM_NVFP4 && (a_tensor_scale || b_tensor_scale)) return GEMM_ERR_INVALID_ARG;
    if (p.M == 0 || p.N == 0) return GEMM_OK;
    if (!C) return GEMM_ERR_INVALID_ARG;
    if (p.K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return GEMM_ERR_INVALID_ARG;
    if ((ep.has_bias != 0) != (bias != nullptr)) return GEMM_ERR_INVALID_ARG;
    if ((ep.has_residual != 0) != (residual != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales))
        return GEMM_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(C) % dtype_size(ep.out_dtype) != 0) return GEMM_ERR_MISALIGNED;
    for (const void* f : {bias, residual, static_cast<const void*>(a_tensor_scale), static_cast<const void*>(b_tensor_scale)})
        if (reinterpret_cast<uintptr_t>(f) % 4 != 0) return GEMM_ERR_MISALIGNED;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess || cur != plan->device) return GEMM_ERR_INVALID_ARG;

    EpiParams e{};
    e.C = C;
    e.ldc = p.ldc;
    e.bias = static_cast<const float*>(bias);
    e.R = static_cast<const float*>(residual);
    e.ldr = ep.ldr;
    e.M = p.M;
    e.N = p.N;
    e.alpha = alpha;
    e.beta = ep.beta;
    e.out_dtype = ep.out_dtype;
    e.act = ep.act;
    LaunchCtx lc{};
    lc.status = plan->d_status;
    lc.timeout_ns = static_cast<uint64_t>(ep.timeout_ms) * 1000000ull;
    lc.flags = ep.flags;
    lc.num_sms = plan->num_sms;
    lc.stream = static_cast<cudaStream_t>(stream);

    const Fp4Operand A{static_cast<const uint8_t*>(a_codes), static_cast<const uint8_t*>(a_scales),
                       a_tensor_scale};
    const Fp4Operand B{static_cast<const uint8_t*>(b_codes), static_cast<const uint8_t*>(b_scales),
                       b_tensor_scale};
    return launch_fp4_gemm(plan->cfg, plan->format, A, B, p.K, e, lc);
}

template <typename P>
int status(P* plan) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    if (cudaDeviceSynchronize() != cudaSuccess) return GEMM_ERR_CUDA;
    unsigned v = 0;
    if (cudaMemcpy(&v, plan->d_status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return (v & 1u) ? GEMM_ERR_DEVICE_TIMEOUT : GEMM_OK;
}

template <typename P>
void destroy(P* plan) {
    {
        std::lock_guard<std::mutex> lk(g_live_mu);
        if (!plan || !live(plan).erase(plan)) return;
    }
    free_plan_memory(plan->d_status);
    delete plan;
}

}  // namespace

extern "C" {

int64_t gemm_fp4_row_bytes(int64_t cols) { return cols < 0 || !sizes_ok(0, cols) ? 0 : fp4_row_bytes(GEMM_MXFP4, cols); }
int64_t gemm_fp8_row_bytes(int64_t cols) { return cols < 0 || !sizes_ok(0, cols) ? 0 : fp4_row_bytes(kMxfp8, cols); }

int64_t gemm_fp4_scales_bytes(gemm_fp4_format_t format, int64_t rows, int64_t cols) {
    return format4(format) ? scales_bytes(format, rows, cols) : 0;
}
int64_t gemm_fp8_scales_bytes(int64_t rows, int64_t cols) { return scales_bytes(kMxfp8, rows, cols); }

int gemm_fp4_quantize(gemm_fp4_format_t format, gemm_dtype_t dtype, int64_t rows, int64_t cols,
                      const void* src, int64_t ld, const float* tensor_scale, void* codes, void* scales,
                      void* stream) {
    if (!format4(format)) return GEMM_ERR_INVALID_ARG;
    return quantize(format, dtype, rows, cols, src, ld, tensor_scale, codes, scales, stream);
}
int gemm_fp8_quantize(gemm_dtype_t dtype, int64_t rows, int64_t cols, const void* src, int64_t ld, void* codes,
                      void* scales, void* stream) {
    return quantize(kMxfp8, dtype, rows, cols, src, ld, nullptr, codes, scales, stream);
}

int gemm_fp4_dequantize(gemm_fp4_format_t format, gemm_dtype_t dtype, int64_t rows, int64_t cols,
                        const void* codes, const void* scales, const float* tensor_scale, void* dst,
                        int64_t ld, void* stream) {
    if (!format4(format)) return GEMM_ERR_INVALID_ARG;
    return dequantize(format, dtype, rows, cols, codes, scales, tensor_scale, dst, ld, stream);
}
int gemm_fp8_dequantize(gemm_dtype_t dtype, int64_t rows, int64_t cols, const void* codes, const void* scales,
                        void* dst, int64_t ld, void* stream) {
    return dequantize(kMxfp8, dtype, rows, cols, codes, scales, nullptr, dst, ld, stream);
}

int gemm_fp4_select_config(int64_t M, int64_t N, int64_t K, int32_t num_sms, gemm_config_t* out) {
    return select_config(GEMM_MXFP4, M, N, K, num_sms, out);
}
int gemm_fp8_select_config(int64_t M, int64_t N, int64_t K, int32_t num_sms, gemm_config_t* out) {
    return select_config(kMxfp8, M, N, K, num_sms, out);
}

int gemm_fp4_plan(gemm_fp4_format_t format, int64_t M, int64_t N, int64_t K, int64_t ldc,
                  const gemm_epilogue_t* epilogue, gemm_fp4_plan_t* out_plan) {
    if (!out_plan) return GEMM_ERR_INVALID_ARG;
    *out_plan = nullptr;
    if (!format4(format)) return GEMM_ERR_INVALID_ARG;
    return make_plan(format, M, N, K, ldc, epilogue, out_plan);
}
int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int64_t ldc, const gemm_epilogue_t* epilogue,
                  gemm_fp8_plan_t* out_plan) {
    if (!out_plan) return GEMM_ERR_INVALID_ARG;
    *out_plan = nullptr;
    return make_plan(kMxfp8, M, N, K, ldc, epilogue, out_plan);
}

int gemm_fp4_run(gemm_fp4_plan_t plan, const void* a_codes, const void* a_scales,
                 const float* a_tensor_scale, const void* b_codes, const void* b_scales,
                 const float* b_tensor_scale, void* C, const void* bias, const void* residual, float alpha,
                 void* stream) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    return run(plan, a_codes, a_scales, a_tensor_scale, b_codes, b_scales, b_tensor_scale, C, bias, residual, alpha,
               stream);
}
int gemm_fp8_run(gemm_fp8_plan_t plan, const void* a_codes, const void* a_scales, const void* b_codes,
                 const void* b_scales, void* C, const void* bias, const void* residual, float alpha, void* stream) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    return run(plan, a_codes, a_scales, nullptr, b_codes, b_scales, nullptr, C, bias, residual, alpha, stream);
}

int gemm_fp4_status(gemm_fp4_plan_t plan) { return status(plan); }
int gemm_fp8_status(gemm_fp8_plan_t plan) { return status(plan); }

void gemm_fp4_destroy(gemm_fp4_plan_t plan) { destroy(plan); }
void gemm_fp8_destroy(gemm_fp8_plan_t plan) { destroy(plan); }

}  // extern "C"
