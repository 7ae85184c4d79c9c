// fp4_gemm.h -- the microscaled 4-bit kernels' launchers and the choice of the
// product's tile (host side).
#pragma once
#include <cstdint>

#include "internal.h"

namespace g13 {

struct Fp4Config {
    int bn;      // tokens per tile: 16, 32, 64, 128, or 256 on CTA pairs
    int splits;  // CTAs of a cluster that share a tile's K (1 to 8)
};
Fp4Config fp4_choose(int fmt, int64_t M, int64_t N, int64_t K, int num_sms);

// A matrix in 4 bits (device pointers).
struct Fp4Operand {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* tensor_scale;  // or null
};

// A: tokens [e.M][K], B: weights [e.N][K]; returns a gemm_status_t.
int launch_fp4_gemm(const Fp4Config& c, int fmt, const Fp4Operand& A, const Fp4Operand& B, int64_t K,
                    const EpiParams& e, const LaunchCtx& lc);
cudaError_t launch_fp4_quantize(int fmt, int dtype, const void* src, int64_t rows, int64_t cols, int64_t ld,
                                const float* g, uint8_t* codes, uint8_t* scales, cudaStream_t st);
cudaError_t launch_fp4_dequantize(int fmt, int dtype, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, void* dst, int64_t rows, int64_t cols, int64_t ld,
                                  cudaStream_t st);

}  // namespace g13
