// w4.cuh -- what the kernels of the 4-bit weights share.
#pragma once
#include <algorithm>

#include "epilogue.cuh"
#include "gelu.cuh"
#include "w4.h"

namespace g13 {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kW4Smem = 226 * 1024;  // at most, of the 227 KB that a CTA can have

// Loads that are made only if `on`, else v keeps what it holds.  (The predicate sits inside the assembly: behind a
// branch the loaded values were copied where the branches meet, which waits for them there.)
__device__ __forceinline__ void ld_codes(uint4& v, const uint8_t* p, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "l"(p), "r"(static_cast<int>(on)));
}
__device__ __forceinline__ void ld_nc32(uint32_t& v, const uint32_t* p, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                 : "+r"(v)
                 : "l"(p), "r"(static_cast<int>(on)));
}
__device__ __forceinline__ void ld_nc16(uint32_t& v, const uint16_t* p, bool on) {  // (into a 32-bit register's low half)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
                 : "+r"(v)
                 : "l"(p), "r"(static_cast<int>(on)));
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ const uint16_t kEights = 0x0808;

// Columns [col, col + 4) of a row's sums through the epilogue (epi_store4's, but for the activations: GELU keeps its
// digits in the left tail, and ReLU of a NaN is NaN, since these kernels have no status word and a NaN is all that tells
// of a wait that ran out).
__device__ __forceinline__ void w4_store4(const EpiParams& e, int64_t row, int64_t col, const float4& v) {
    if (row >= e.M || col >= e.N) return;
    float y[4] = {v.x * e.alpha, v.y * e.alpha, v.z * e.alpha, v.w * e.alpha};
    if (e.bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j < e.N) y[j] += __ldg(e.bias + col + j);
    }
    if (e.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = y[j] < 0.0f ? 0.0f : y[j];
    } else if (e.act == GEMM_ACT_GELU_ERF) {
        gelu2(y[0], y[1]);
        gelu2(y[2], y[3]);
    }
    EpiParams rest = e;  // the residual and the cast
    rest.alpha = 1.0f;
    rest.bias = nullptr;
    rest.act = GEMM_ACT_NONE;
    epi_store4(rest, 0, row, col, y[0], y[1], y[2], y[3]);
}

// The groups that a step meets: one, two, or four (of which some may be the same one).
__host__ __device__ constexpr int w4_per_step(int64_t group) { return group % 128 == 0 ? 1 : group % 64 == 0 ? 2 : 4; }

// i / n by n's reciprocal.
__device__ __forceinline__ int over(uint32_t i, uint32_t inv) { return static_cast<int>(inv ? __umulhi(i, inv) : i); }
inline uint32_t reciprocal(int64_t n) {
    return n == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + static_cast<uint64_t>(n) - 1) / static_cast<uint64_t>(n));
}

// Clusters of `splits` CTAs that run at a time, with one CTA to an SM: a cluster stays within a part of the GPU, so
// the larger ones leave SMs over (152 SMs hold 76, 36 and 15 of 2, 4 and 8).
inline int64_t clusters_at_once(int splits, int num_sms) {
    return splits == 1 ? num_sms : splits == 2 ? num_sms / 2 : splits == 4 ? num_sms / 4 - num_sms / 76 : num_sms / 10;
}

}  // namespace
}  // namespace g13
