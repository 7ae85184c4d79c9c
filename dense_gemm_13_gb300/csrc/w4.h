// w4.h -- 4-bit weights with group scales: layout, sizes and launchers.
//
// Codes lie in blocks of 16 rows x 64 columns, 512 bytes each: what a warp loads at once, 16 bytes a lane,
// as the fragments of four matrix instructions of 16 x 16.  Lane 4 (r % 8) + k % 32 / 8 has the words of rows
// r and r + 8 for the block's first 32 columns, then for its last; a word's eight columns lie so that
// (word >> 4 i) & 0x000F000F is columns 2 i and 2 i + 1.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

#ifdef __CUDACC__
#define G13_W4_HD __host__ __device__
#else
#define G13_W4_HD
#endif

namespace g13 {

constexpr int64_t kW4MaxTokens = 64, kW4MaxK = 65536, kW4MaxN = int64_t(1) << 28;

G13_W4_HD inline constexpr int64_t w4_tiles(int64_t N) { return (N + 15) / 16; }
G13_W4_HD inline constexpr int64_t w4_blocks(int64_t K) { return (K + 63) / 64; }
G13_W4_HD inline constexpr int64_t w4_groups(int64_t K, int64_t group) { return (K + group - 1) / group; }
// The 32-bit word that holds columns k .. k + 7 (k a multiple of 8) of row r.
G13_W4_HD inline constexpr int64_t w4_word(int64_t r, int64_t k, int64_t blocks) {
    return (r / 16 * blocks + k / 64) * 128 + ((r % 8) * 4 + k % 32 / 8) * 4 + k % 64 / 32 * 2 + r % 16 / 8;
}
// The entry of row r, group c in the arrays of scales and zeros.
G13_W4_HD inline constexpr int64_t w4_entry(int64_t r, int64_t c, int64_t groups) {
    return (r / 16 * groups + c) * 16 + r % 8 * 2 + r % 16 / 8;
}

struct W4Args {
    int dtype;  // X and scales: GEMM_F16 or GEMM_BF16
    int64_t M, N, K, group, ldx;
    const void* x;
    const uint8_t* codes;
    const void* scales;
    const uint8_t* zeros;  // or null: 8
    EpiParams e;
    uint64_t timeout_ns;  // of the waits inside a kernel
    uint32_t flags;
};

// How a product is cut: 8 * nt tokens a pass, `splits` CTAs of a cluster to K, `wk` of a CTA's warps to its part of K.
struct W4Config {
    int nt, splits, wk;
};
W4Config w4_choose(int64_t M, int64_t N, int64_t K, int64_t group, int num_sms);

cudaError_t launch_w4(const W4Config& c, const W4Args& a, int num_sms, cudaStream_t st);
// On the tensor cores: into how many CTAs of a cluster K is divided, 0 where launch_w4 is better (or X is not aligned).
int w4_tc_splits(const W4Args& a, int num_sms);
cudaError_t launch_w4_tc(const W4Args& a, int splits, cudaStream_t st);
// src: [N][ld] of `dtype`; scales of `scale_dtype`; zeros null: symmetric.
cudaError_t launch_w4_quantize(int dtype, int scale_dtype, int64_t N, int64_t K, int64_t group, const void* src,
                               int64_t ld, uint8_t* codes, void* scales, uint8_t* zeros, cudaStream_t st);
// One byte a code, scales and zeros in rows, to the layout above.
cudaError_t launch_w4_pack(int64_t N, int64_t K, int64_t group, const uint8_t* q, int64_t ldq,
                           const void* s, int64_t lds, const uint8_t* z, int64_t ldz, uint8_t* codes, void* scales,
                           uint8_t* zeros, cudaStream_t st);
cudaError_t launch_w4_dequantize(int dtype, int scale_dtype, int64_t N, int64_t K, int64_t group,
                                 const uint8_t* codes, const void* scales, const uint8_t* zeros, void* dst,
                                 int64_t ld, cudaStream_t st);

}  // namespace g13
