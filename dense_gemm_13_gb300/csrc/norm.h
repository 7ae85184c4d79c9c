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

// How a row lies in its threads' chunks of eight elements.
enum NormLay {
    SINGLES = 0,  // element i of a chunk is i * (threads of a row) columns on
    ALIGNED = 1,  // eight neighbours, the first chunk at column 0
    PHASED = 2    // eight neighbours, the first chunk at column -o, 0 <= o < 8
};

// Phased rows go up to this many columns: what is moved fits the shared memory, or a row the registers.
constexpr int norm_phased(bool f8) { return f8 ? 8192 - 7 : 16384 - 7; }

struct NormShape {
    int cols;
    Two inv;                 // 1 / cols
    int64_t rows, rows_all;  // rows_all: with the padding of the scales' last tile
    int64_t row_bytes, col_tiles;
    int phase, phase_step;   // by how many elements row 0 is off 16 bytes, and each row more (of eight; FP32 alone: of four)
    NormLay lay;
    bool wide_weight;        // the weight takes loads of eight 16-bit numbers
};

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st);
// The kernels, a file each: any types, or rows and residual of one 16-bit type.
cudaError_t launch_norm_any(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);
cudaError_t launch_norm_bf16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);
cudaError_t launch_norm_f16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);
cudaError_t launch_norm8_any(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);
cudaError_t launch_norm8_bf16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);
cudaError_t launch_norm8_f16(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st);

}  // namespace g13
