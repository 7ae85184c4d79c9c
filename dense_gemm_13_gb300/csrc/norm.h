// norm.h -- root-mean-square norm: arguments and launcher.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "gemm13.h"

namespace g13 {

constexpr int64_t kNormMaxCols = int64_t(1) << 22;

struct NormArgs {
    gemm_norm_desc_t d;
    const void* x;
    const void* r;  // residual, or null
    const void* w;  // or null
    void* h;        // or null
    void* y;        // values, or codes
    uint8_t* scales;
};

// A number as the sum of two, the second of them what the first leaves.
struct Two {
    float hi, lo;
};

struct NormShape {
    int cols;
    Two inv;                 // 1 / cols
    int64_t rows, rows_all;  // rows_all: with the padding of the scales' last tile
    int64_t row_bytes, col_tiles;
    int phase, phase_step;   // by how many elements row 0 is off 16 bytes, and each row more (of eight; FP32 alone: of four)
    bool wide_weight;        // the weight takes loads of eight 16-bit numbers
};

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st);

}  // namespace g13
