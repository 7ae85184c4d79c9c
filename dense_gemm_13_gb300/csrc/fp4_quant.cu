// fp4_quant.cu -- matrices to microscaled 4-bit (and 8-bit) floats and back.
//
//   mxfp4  d = 2^E, E = floor(log2 max|x|) - 2 over blocks of 32, kept in
//          [-127, 127] (the exponent rule of the OCP microscaling formats)
//   nvfp4  s = E4M3(max|x| / (6 g)) over blocks of 16, d = fl32(s g), with a
//          scale g of the whole tensor
//   code   = nearest E2M1 value to fl32(x / d), ties to even, saturating at 6
//   mxfp8  blocks of 32 as mxfp4's, E the least with max|x| <= 448 2^E (mxfp4's rule would
//          saturate the largest eighth of a binade); code = nearest E4M3 value to x / d
//
// Both directions move every byte once, so memory bounds them.  A thread takes
// 16 elements at a time (an nvfp4 block; half an mxfp4 block, joined by one
// shuffle): 32 bytes of 16-bit input, 8 bytes of codes.  The scale bytes of a row
// are 512 bytes apart in the stored tiles; a quantising CTA therefore takes the 32
// rows r, r + 32, r + 64, r + 96 (r = 8 consecutive rows) that share 128
// consecutive bytes of a tile, gathers their scales in shared memory and
// writes whole sectors.  Rows that are not 16-byte aligned go through shared
// memory, so that global accesses stay coalesced.
// Measured on 8192 x 8192 (bytes of both sides over time): quantising FP32 6.6 TB/s,
// BF16 6.2 (mxfp4) and 4.9 (nvfp4: 15 instructions an element, latency at 64 warps per SM;
// 40 us instead of 35 at 4 CTAs per SM), reading back 6.6 (FP32) and 6.0 (BF16).  The FP32
// form holds 5 CTAs per SM (at 8 its 32 loaded registers spill: 68 us instead of 46).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8.cuh"
#include "internal.h"

namespace g13 {
namespace {

constexpr int QT = 256;       // threads per CTA
constexpr int QCOLS = 256;    // columns that a CTA's threads take at a time
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

// 16 consecutive elements of a row.
template <typename T>
struct __align__(16) Sixteen {
    T v[16];
};
// Of which n exist (the rest are zero); 16-byte loads where all do.
template <typename T>
__device__ __forceinline__ Sixteen<T> load16(const T* p, int64_t n) {
    Sixteen<T> x;
    if (n >= 16) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
            reinterpret_cast<uint4*>(x.v)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x.v[i] = i < n ? p[i] : from_f32<T>(0.0f);
    }
    return x;
}

// The largest magnitude as the bits of an FP32 number; infinities and NaN compare above
// every number.
__device__ __forceinline__ uint32_t top16(const Sixteen<float>& x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x.v[i]) & 0x7FFFFFFFu);
    return m;
}
template <typename T, typename T2>
__device__ __forceinline__ uint32_t top16_packed(const Sixteen<T>& x) {
    const T2* p = reinterpret_cast<const T2*>(x.v);
    T2 m = __habs2(p[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(p[i]));
    return max(__float_as_uint(to_f32<T>(m.x)) & 0x7FFFFFFFu, __float_as_uint(to_f32<T>(m.y)) & 0x7FFFFFFFu);
}
__device__ __forceinline__ uint32_t top16(const Sixteen<__half>& x) { return top16_packed<__half, __half2>(x); }
__device__ __forceinline__ uint32_t top16(const Sixteen<__nv_bfloat16>& x) {
    return top16_packed<__nv_bfloat16, __nv_bfloat162>(x);
}
// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// VEC: rows are 16-byte aligned.
template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(QT, sizeof(T) == 4 ? 5 : FMT == kMxfp8 ? 6 : 8)
    fp4_quantize_kernel(const T* __restrict__ src, int64_t rows, int64_t cols, int64_t ld,
                        const float* __restrict__ gscale, uint8_t* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t col_blocks) {
    constexpr int BLK = fp4_block(FMT);
    constexpr int TILES = QCOLS / (4 * BLK);      // scale tiles along the CTA's columns
    constexpr int LINE = QCOLS + 16 / sizeof(T);  // a staged row
    __shared__ __align__(16) uint8_t sc[TILES][128];
    __shared__ __align__(16) T stage[VEC ? 1 : QROWS * LINE];
    const int64_t rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int64_t rt = rb >> 2;          // row tile of 128
    const int sub = static_cast<int>(rb & 3);
    const int64_t row_bytes = fp4_row_bytes(FMT, cols);
    const int64_t ctiles = fp4_col_tiles(FMT, cols);
    const float g = FMT == GEMM_NVFP4 && gscale ? __ldg(gscale) : 1.0f;
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
    // slot 0..31 of the CTA -> row
    const auto row_of = [&](int slot) { return rt * 128 + (slot >> 3) * 32 + sub * 8 + (slot & 7); };

    Sixteen<T> x[2];
    if constexpr (VEC) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int64_t row = row_of(p * 16 + tr), c0 = cb * QCOLS + tc * 16;
            x[p] = load16<T>(src + row * ld + c0, row < rows ? cols - c0 : 0);
        }
    } else {
        const int64_t c = cb * QCOLS + threadIdx.x;
#pragma unroll
        for (int i = 0; i < QROWS; ++i) {
            const int64_t row = row_of(i);
            stage[i * LINE + threadIdx.x] = row < rows && c < cols ? src[row * ld + c] : from_f32<T>(0.0f);
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 2; ++p)
            x[p] = *reinterpret_cast<const Sixteen<T>*>(&stage[(p * 16 + tr) * LINE + tc * 16]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int slot = p * 16 + tr;
        const int64_t row = row_of(slot), c0 = cb * QCOLS + tc * 16;
        uint32_t top = top16(x[p]);
        if (BLK == 32) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        uint32_t byte;
        float d = 1.0f, inv;
        bool near = true;  // the block's quotients x / d stay far inside FP32
        if (FMT == GEMM_MXFP4) {
            // floor(log2) of a normal number is its exponent field; below the
            // normal range the result is kept at -127 anyway
            const int e = static_cast<int>(top >> 23) - 127 - 2;
            byte = top >= 0x7F800000u ? 0xFFu : static_cast<uint32_t>(max(e, -127) + 127);
            inv = ue8m0_value(254u - min(byte, 254u));  // 2^-E
        } else if (FMT == kMxfp8) {
            byte = mxfp8_scale(top);
            inv = ue8m0_value(254u - min(byte, 254u));
        } else {
            const float r = __fdiv_rn(__uint_as_float(top), 6.0f * g);
            near = r < 0x1p60f;
            byte = top >= 0x7F800000u ? 0x7Fu : e4m3_byte(fminf(r, 448.0f));
            d = e4m3_value(byte) * g;
            inv = __frcp_rn(d);
        }
        uint32_t code[FMT == kMxfp8 ? 4 : 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(x[p].v[8 * h + i]);
            if (BLK == 32) {
                // exact products, apart from results far below the least code
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
            } else if (d > 0x1p-60f && d < 0x1p60f && near) {
                // fl32(x / d): q = x (1/d) corrected by its exact remainder, which gives the
                // rounded quotient (P. Markstein, "Computation of elementary functions on the
                // IBM RISC System/6000 processor", 1990) as long as q is finite; one and a half
                // instructions an element where a division each would take longer than the memory
                const uint64_t inv2 = pack2(inv, inv), nd2 = pack2(-d, -d);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint64_t v2 = pack2(v[i], v[i + 1]), q = mul2(v2, inv2);
                    const uint64_t r = fma2(fma2(q, nd2, v2), inv2, q);
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(y[i]), "=f"(y[i + 1]) : "l"(r));
                    // (the remainder of -0 is +0: the sign is put back)
                    y[i] = copysignf(y[i], v[i]);
                    y[i + 1] = copysignf(y[i + 1], v[i + 1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = d > 0.0f ? __fdiv_rn(v[i], d) : 0.0f * v[i];
            }
            if constexpr (FMT == kMxfp8) {
                code[2 * h] = e4m3x4(y);
                code[2 * h + 1] = e4m3x4(y + 4);
            } else {
                code[h] = e2m1x8(y);
            }
        }
        if constexpr (FMT == kMxfp8) {
            if (row < rows && c0 < row_bytes)
                *reinterpret_cast<uint4*>(codes + row * row_bytes + c0) = make_uint4(code[0], code[1], code[2], code[3]);
        } else {
            if (row < rows && c0 / 2 < row_bytes)
                *reinterpret_cast<uint2*>(codes + row * row_bytes + c0 / 2) = make_uint2(code[0], code[1]);
        }
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

// One thread per 16 elements.  ALIGN: bytes that every row of dst starts on (32: whole
// sectors per store; 16; else through shared memory, 32 neighbouring elements a store).
template <int FMT, typename T, int ALIGN>
__global__ void __launch_bounds__(QT)
    fp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                          const float* __restrict__ gscale, T* __restrict__ dst, int64_t rows,
                          int64_t cols, int64_t ld, int64_t groups) {
    __shared__ __align__(16) T stage[ALIGN >= 16 ? 1 : QT * 16];
    const int64_t i = static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x;
    const int64_t row = i / groups;
    const int64_t c0 = (i - row * groups) * 16;
    __align__(32) T out[16];
    if (row < rows) {
        const int64_t row_bytes = fp4_row_bytes(FMT, cols);
        const int64_t blk = c0 / fp4_block(FMT);
        const int r = static_cast<int>(row & 127);
        const uint32_t byte =
            __ldg(scales + ((row >> 7) * fp4_col_tiles(FMT, cols) + (blk >> 2)) * kFp4TileBytes +
                  (r & 31) * 16 + (r >> 5) * 4 + (blk & 3));
        const float d = fp4_block(FMT) == 32 ? ue8m0_value(byte)
                                             : e4m3_value(byte) * (gscale ? __ldg(gscale) : 1.0f);
        float y[16];
        if constexpr (FMT == kMxfp8) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + row * row_bytes + c0));
            e4m3x4_values(w.x, y);
            e4m3x4_values(w.y, y + 4);
            e4m3x4_values(w.z, y + 8);
            e4m3x4_values(w.w, y + 12);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + row * row_bytes + c0 / 2));
            e2m1x8_values(w.x, y);
            e2m1x8_values(w.y, y + 8);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) out[j] = from_f32<T>(y[j] * d);
    }
    if constexpr (ALIGN >= 16) {
        if (row >= rows) return;
        T* p = dst + row * ld + c0;
        const uint32_t* o = reinterpret_cast<const uint32_t*>(out);
        if (c0 + 16 <= cols) {
            if constexpr (ALIGN == 32) {
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                     reinterpret_cast<char*>(p) + 32 * j),
                                 "r"(o[8 * j]), "r"(o[8 * j + 1]), "r"(o[8 * j + 2]), "r"(o[8 * j + 3]),
                                 "r"(o[8 * j + 4]), "r"(o[8 * j + 5]), "r"(o[8 * j + 6]), "r"(o[8 * j + 7])
                                 : "memory");
            } else {
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)); ++j)
                    reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<const uint4*>(out)[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c0 + j < cols) p[j] = out[j];
        }
    } else {
        // a warp's 32 groups: element j of the warp's 512 by lane j % 32
        const int lane = threadIdx.x & 31;
        T* mine = stage + (threadIdx.x >> 5) * 512;
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(T)); ++j)
            reinterpret_cast<uint4*>(mine + lane * 16)[j] = reinterpret_cast<const uint4*>(out)[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            // the group that element 32 j + lane belongs to, as its thread sees it
            const int src = 2 * j + (lane >> 4);
            const int64_t r = __shfl_sync(0xFFFFFFFFu, row, src);
            const int64_t c = __shfl_sync(0xFFFFFFFFu, c0, src) + (lane & 15);
            if (r < rows && c < cols) dst[r * ld + c] = mine[32 * j + lane];
        }
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
    const auto on = [&](uintptr_t n) { return reinterpret_cast<uintptr_t>(dst) % n == 0 && ld * sizeof(T) % n == 0; };
    const int64_t groups = (cols + 15) / 16;
    const int64_t grid = (rows * groups + QT - 1) / QT;
    auto k = on(32)   ? fp4_dequantize_kernel<FMT, T, 32>
             : on(16) ? fp4_dequantize_kernel<FMT, T, 16>
                      : fp4_dequantize_kernel<FMT, T, 0>;
    k<<<static_cast<unsigned>(grid), QT, 0, st>>>(codes, scales, g, static_cast<T*>(dst), rows, cols, ld,
                                                  groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, int dtype, const void* src, int64_t rows, int64_t cols,
                                int64_t ld, const float* g, uint8_t* codes, uint8_t* scales,
                                cudaStream_t st) {
    const auto run = [&](auto f) {
        constexpr int F = decltype(f)::value;
        if (dtype == GEMM_F32) return quantize_t<F, float>(src, rows, cols, ld, g, codes, scales, st);
        if (dtype == GEMM_F16) return quantize_t<F, __half>(src, rows, cols, ld, g, codes, scales, st);
        return quantize_t<F, __nv_bfloat16>(src, rows, cols, ld, g, codes, scales, st);
    };
    if (fmt == kMxfp8) return run(std::integral_constant<int, kMxfp8>{});
    if (fmt == GEMM_MXFP4) return run(std::integral_constant<int, GEMM_MXFP4>{});
    return run(std::integral_constant<int, GEMM_NVFP4>{});
}

cudaError_t launch_fp4_dequantize(int fmt, int dtype, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, void* dst, int64_t rows, int64_t cols, int64_t ld,
                                  cudaStream_t st) {
    const auto run = [&](auto f) {
        constexpr int F = decltype(f)::value;
        if (dtype == GEMM_F32) return dequantize_t<F, float>(codes, scales, g, dst, rows, cols, ld, st);
        if (dtype == GEMM_F16) return dequantize_t<F, __half>(codes, scales, g, dst, rows, cols, ld, st);
        return dequantize_t<F, __nv_bfloat16>(codes, scales, g, dst, rows, cols, ld, st);
    };
    if (fmt == kMxfp8) return run(std::integral_constant<int, kMxfp8>{});
    if (fmt == GEMM_MXFP4) return run(std::integral_constant<int, GEMM_MXFP4>{});
    return run(std::integral_constant<int, GEMM_NVFP4>{});
}

}  // namespace g13
