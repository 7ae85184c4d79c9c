// fp8.cuh -- E4M3 values and UE8M0 scales, as the kernels that write or read them convert.
#pragma once
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace g13 {
namespace {

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

// Four FP32 values to E4M3 bytes, the first in the lowest (round to nearest even, at most 448 in magnitude).
__device__ __forceinline__ uint32_t e4m3x4(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return r;
}
// Four E4M3 bytes to FP32.
__device__ __forceinline__ void e4m3x4_values(uint32_t codes, float* y) {
    uint32_t h[2];
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}
// The scale byte of an mxfp8 block whose largest magnitude has the FP32 bits `top`: exponent E + 127, E the
// least with max <= 448 * 2^E = 1.75 * 2^(E + 8), kept in [-127, 127]; 255 (NaN) where top is an infinity or a NaN.
__device__ __forceinline__ uint32_t mxfp8_scale(uint32_t top) {
    if (top >= 0x7F800000u) return 0xFFu;
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(max(e, -127) + 127);
}

}  // namespace
}  // namespace g13
