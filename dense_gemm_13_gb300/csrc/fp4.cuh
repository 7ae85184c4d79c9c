// fp4.cuh -- the microscaled formats: constants and the layout of the stored
// scales, shared by the quantisation kernels and the block-scaled products.
//
// A matrix in 4 bits is two arrays.  Codes: E2M1 values, two to a byte (the
// first in the low half), rows of fp4_row_bytes() bytes, padded with zeros.
// Scales: one byte per block of a row, in tiles of 128 rows x 4 blocks (512
// bytes): row r, block c of a tile at byte (r % 32) * 16 + (r / 32) * 4 + c,
// tiles along a row of tiles first.  That order is the one in which
// tcgen05.mma reads block scales from TMEM -- 32 lanes x 16 bytes, the four
// groups of 32 rows side by side -- so a tile goes from global memory to
// shared memory to TMEM in two straight copies.
//
// mxfp8 (kMxfp8) is the same with E4M3 values, a byte each, in rows padded to 32
// elements, and blocks of 32 with scales as mxfp4's.
#pragma once
#include <cstdint>

#include "gemm13.h"

#ifdef __CUDACC__
#define G13_HD __host__ __device__
#else
#define G13_HD
#endif

namespace g13 {

constexpr int kMxfp8 = 2;  // beside gemm_fp4_format_t's values

G13_HD inline constexpr int fp4_block(int fmt) { return fmt == GEMM_NVFP4 ? 16 : 32; }
G13_HD inline constexpr int64_t fp4_row_bytes(int fmt, int64_t cols) {
    return (cols + 31) / 32 * (fmt == kMxfp8 ? 32 : 16);
}
// K elements of a 128-byte piece of a row: what a stage of the product's ring holds.
G13_HD inline constexpr int fp4_stage_k(int fmt) { return fmt == kMxfp8 ? 128 : 256; }
G13_HD inline constexpr int64_t fp4_row_tiles(int64_t rows) { return (rows + 127) / 128; }
// Tiles of four blocks along a row.
G13_HD inline constexpr int64_t fp4_col_tiles(int fmt, int64_t cols) {
    return (cols + 4 * fp4_block(fmt) - 1) / (4 * fp4_block(fmt));
}
constexpr int kFp4TileBytes = 512;

}  // namespace g13
