// fp4_quant.cu -- matrices to microscaled 4-bit floats and back.
//
//   mxfp4  d = 2^E, E = floor(log2 max|x|) - 2 over blocks of 32, kept in
//          [-127, 127] (the exponent rule of the OCP microscaling formats)
//   nvfp4  s = E4M3(max|x| / (6 g)) over blocks of 16, d = fl32(s g), with a
//          scale g of the whole tensor
//   code   = nearest E2M1 value to fl32(x / d), ties to even, saturating at 6
//
// Both directions move every byte once, so memory bounds them.  A thread takes
// 16 elements (an nvfp4 block; half an mxfp4 block, joined by one shuffle):
// 32 bytes of 16-bit input, 8 bytes of codes.  The scale bytes of a row are
// 512 bytes apart in the stored tiles; a quantising CTA therefore takes the 32
// rows r, r + 32, r + 64, r + 96 (r = 8 consecutive rows) that share 128
// consecutive bytes of a tile, gathers their scales in shared memory and
// writes whole sectors.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "internal.h"

namespace g13 {
namespace {

constexpr int QT = 256;       // threads per CTA
constexpr int QCOLS = 256;    // columns per quantising CTA
constexpr int QROWS = 32;     // rows per quantising CTA

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// Eight FP32 values to eight E2M1 codes, the first in the lowest four bits
// (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e2m1x8(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// Eight codes to FP32.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float* y) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}

// E4M3 byte of a value in [0, 448] (round to nearest even), and its value.
__device__ __forceinline__ uint32_t e4m3_byte(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}
// The value of a UE8M0 byte, 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
    if (byte == 0xFFu) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// 16 consecutive elements as FP32: 16-byte loads, or (VEC false, or the row's
// end) one by one with zeros past `n`.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T* p, int64_t n, float* x) {
    if (VEC && n >= 16) {
        constexpr int W = 16 / sizeof(T);
        uint4 v[16 / W];
#pragma unroll
        for (int i = 0; i < 16 / W; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = to_f32<T>(reinterpret_cast<const T*>(v)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i < n ? to_f32<T>(p[i]) : 0.0f;
    }
}

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(QT)
    fp4_quantize_kernel(const T* __restrict__ src, int64_t rows, int64_t cols, int64_t ld,
                        const float* __restrict__ gscale, uint8_t* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t col_blocks) {
    constexpr int BLK = fp4_block(FMT);
    constexpr int TILES = QCOLS / (4 * BLK);  // scale tiles along the CTA's columns
    __shared__ __align__(16) uint8_t sc[TILES][128];
    const int64_t rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int64_t rt = rb >> 2;          // row tile of 128
    const int sub = static_cast<int>(rb & 3);
    const int64_t row_bytes = fp4_row_bytes(cols);
    const int64_t ctiles = fp4_col_tiles(FMT, cols);
    const float g = FMT == GEMM_NVFP4 && gscale ? __ldg(gscale) : 1.0f;
    const int tc = threadIdx.x & 15;
    const int64_t c0 = cb * QCOLS + tc * 16;

    float x[2][16];
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const int slot = pass * 16 + (threadIdx.x >> 4);
        const int64_t row = rt * 128 + (slot >> 3) * 32 + sub * 8 + (slot & 7);
        load16<T, VEC>(src + row * ld + c0, row < rows ? cols - c0 : 0, x[pass]);
    }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const int slot = pass * 16 + (threadIdx.x >> 4);
        const int64_t row = rt * 128 + (slot >> 3) * 32 + sub * 8 + (slot & 7);
        // the largest magnitude as bits: infinities and NaN compare above every number
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[pass][i]) & 0x7FFFFFFFu);
        if (FMT == GEMM_MXFP4) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        uint32_t byte;
        float y[16];
        if (FMT == GEMM_MXFP4) {
            // floor(log2) of a normal number is its exponent field; below the
            // normal range the result is kept at -127 anyway
            const int e = static_cast<int>(top >> 23) - 127 - 2;
            byte = top >= 0x7F800000u ? 0xFFu : static_cast<uint32_t>(max(e, -127) + 127);
            // 2^-E; exact products, apart from results far below the least code
            const float inv = ue8m0_value(254u - min(byte, 254u));
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = x[pass][i] * inv;
        } else {
            const float r = fminf(__fdiv_rn(__uint_as_float(top), 6.0f * g), 448.0f);
            byte = top >= 0x7F800000u ? 0x7Fu : e4m3_byte(r);
            const float d = e4m3_value(byte) * g;
            if (d > 0x1p-60f && d < 0x1p60f) {
                // fl32(x / d): q = x (1/d) corrected by its exact remainder, which gives the
                // rounded quotient (P. Markstein, "Computation of elementary functions on the
                // IBM RISC System/6000 processor", 1990); three operations an element where
                // a division each would take longer than the memory
                const float inv = __frcp_rn(d);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float q = x[pass][i] * inv;
                    // (the remainder of -0 is +0: the sign is put back)
                    y[i] = copysignf(fmaf(fmaf(-q, d, x[pass][i]), inv, q), x[pass][i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = d > 0.0f ? __fdiv_rn(x[pass][i], d) : 0.0f * x[pass][i];
            }
        }
        if (row < rows && c0 / 2 < row_bytes)
            *reinterpret_cast<uint2*>(codes + row * row_bytes + c0 / 2) =
                make_uint2(e2m1x8(y), e2m1x8(y + 8));
        // blocks past the row's end and rows past the matrix: zeros
        if (row >= rows || c0 / BLK >= (cols + BLK - 1) / BLK) byte = 0;
        const int blk = tc * 16 / BLK;  // block within the CTA
        if (FMT == GEMM_NVFP4 || (tc & 1) == 0)
            sc[blk >> 2][(slot & 7) * 16 + (slot >> 3) * 4 + (blk & 3)] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < TILES * 8 && cb * TILES + (t >> 3) < ctiles)
        *reinterpret_cast<uint4*>(scales + (rt * ctiles + cb * TILES + (t >> 3)) * kFp4TileBytes +
                                  sub * 128 + (t & 7) * 16) =
            *reinterpret_cast<const uint4*>(&sc[t >> 3][(t & 7) * 16]);
}

// One thread per 16 elements.
template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(QT)
    fp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                          const float* __restrict__ gscale, T* __restrict__ dst, int64_t rows,
                          int64_t cols, int64_t ld, int64_t groups) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x;
    const int64_t row = i / groups;
    if (row >= rows) return;
    const int64_t c0 = (i - row * groups) * 16;
    const int64_t row_bytes = fp4_row_bytes(cols);
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + row * row_bytes + c0 / 2));
    const int64_t blk = c0 / fp4_block(FMT);
    const int r = static_cast<int>(row & 127);
    const uint32_t byte = __ldg(scales + ((row >> 7) * fp4_col_tiles(FMT, cols) + (blk >> 2)) * kFp4TileBytes +
                                (r & 31) * 16 + (r >> 5) * 4 + (blk & 3));
    const float d = FMT == GEMM_MXFP4 ? ue8m0_value(byte)
                                      : e4m3_value(byte) * (gscale ? __ldg(gscale) : 1.0f);
    float y[16];
    e2m1x8_values(w.x, y);
    e2m1x8_values(w.y, y + 8);
    __align__(16) T out[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) out[j] = from_f32<T>(y[j] * d);
    T* p = dst + row * ld + c0;
    if (VEC && c0 + 16 <= cols) {
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(T)); ++j)
            reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<const uint4*>(out)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c0 + j < cols) p[j] = out[j];
    }
}

template <int FMT, typename T>
cudaError_t quantize_t(const void* src, int64_t rows, int64_t cols, int64_t ld, const float* g,
                       uint8_t* codes, uint8_t* scales, cudaStream_t st) {
    const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && ld * sizeof(T) % 16 == 0;
    const int64_t cbs = (cols + QCOLS - 1) / QCOLS;
    const int64_t grid = fp4_row_tiles(rows) * (128 / QROWS) * cbs;
    auto k = vec ? fp4_quantize_kernel<FMT, T, true> : fp4_quantize_kernel<FMT, T, false>;
    k<<<static_cast<unsigned>(grid), QT, 0, st>>>(static_cast<const T*>(src), rows, cols, ld, g, codes,
                                                  scales, cbs);
    return cudaGetLastError();
}

template <int FMT, typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, const float* g, void* dst,
                         int64_t rows, int64_t cols, int64_t ld, cudaStream_t st) {
    const bool vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0 && ld * sizeof(T) % 16 == 0;
    const int64_t groups = (cols + 15) / 16;
    const int64_t grid = (rows * groups + QT - 1) / QT;
    auto k = vec ? fp4_dequantize_kernel<FMT, T, true> : fp4_dequantize_kernel<FMT, T, false>;
    k<<<static_cast<unsigned>(grid), QT, 0, st>>>(codes, scales, g, static_cast<T*>(dst), rows, cols, ld,
                                                  groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, int dtype, const void* src, int64_t rows, int64_t cols,
                                int64_t ld, const float* g, uint8_t* codes, uint8_t* scales,
                                cudaStream_t st) {
    if (fmt == GEMM_MXFP4) {
        if (dtype == GEMM_F32)
            return quantize_t<GEMM_MXFP4, float>(src, rows, cols, ld, g, codes, scales, st);
        if (dtype == GEMM_F16)
            return quantize_t<GEMM_MXFP4, __half>(src, rows, cols, ld, g, codes, scales, st);
        return quantize_t<GEMM_MXFP4, __nv_bfloat16>(src, rows, cols, ld, g, codes, scales, st);
    }
    if (dtype == GEMM_F32)
        return quantize_t<GEMM_NVFP4, float>(src, rows, cols, ld, g, codes, scales, st);
    if (dtype == GEMM_F16)
        return quantize_t<GEMM_NVFP4, __half>(src, rows, cols, ld, g, codes, scales, st);
    return quantize_t<GEMM_NVFP4, __nv_bfloat16>(src, rows, cols, ld, g, codes, scales, st);
}

cudaError_t launch_fp4_dequantize(int fmt, int dtype, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, void* dst, int64_t rows, int64_t cols, int64_t ld,
                                  cudaStream_t st) {
    if (fmt == GEMM_MXFP4) {
        if (dtype == GEMM_F32)
            return dequantize_t<GEMM_MXFP4, float>(codes, scales, g, dst, rows, cols, ld, st);
        if (dtype == GEMM_F16)
            return dequantize_t<GEMM_MXFP4, __half>(codes, scales, g, dst, rows, cols, ld, st);
        return dequantize_t<GEMM_MXFP4, __nv_bfloat16>(codes, scales, g, dst, rows, cols, ld, st);
    }
    if (dtype == GEMM_F32)
        return dequantize_t<GEMM_NVFP4, float>(codes, scales, g, dst, rows, cols, ld, st);
    if (dtype == GEMM_F16)
        return dequantize_t<GEMM_NVFP4, __half>(codes, scales, g, dst, rows, cols, ld, st);
    return dequantize_t<GEMM_NVFP4, __nv_bfloat16>(codes, scales, g, dst, rows, cols, ld, st);
}

}  // namespace g13
