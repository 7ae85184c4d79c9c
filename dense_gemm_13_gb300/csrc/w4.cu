// w4.cu -- products of a few tokens with 4-bit weights and group scales:
//
//   Y = cast( act( alpha sum_k X[m,k] (q[n,k] - z[n,k/g]) s[n,k/g] + bias[n] ) + beta R[m,n] )
//
// The weights' bytes are the cost (half a byte a weight); every one is read once, by 16-byte loads of whole 512-byte
// blocks, several ahead in registers.  A warp multiplies a step of 16 rows x 128 columns with 8 tokens by eight mma.sync
// m16n8k16: the weights are the 16 rows, the tokens the columns.  What is left to save is instructions, so the codes go into
// the product nearly as they lie: a nibble in the second lowest place of 16 bits, the others masked off, is the FP16
// number 16 q 2^-24, exactly (its subnormal range is linear).  Seven instructions make eight weights (as 1024 + q or 128 + q,
// minus 1024 + z: nine and eleven).  In the lowest place two less would do, but the tensor cores line their sums up as if a
// subnormal were 2^-14, and cut off what a small one has too far down: K = 8192, FP16, FP32 results 1.6e-6 of them off
// instead of 1.8e-7 (16 tokens 30.8 us instead of 31.5, 1 x 16384 x 8192 16.9 instead of 17.6).  The zero comes off afterwards:
//
//   sum_k (q - z) x = sum_k q x - z sum_k x      over a group, FP32; the sums of x are worked out once per CTA
//
// and the group's scale multiplies the difference, so no weight is rounded.  The activations are brought into the upper
// part of FP16's range by a power of two for every 128 of a token's: exact, but for values below 2^-31 of the largest of them
// (FP16 ones: 2^-28), which are off by 2^-39 of it at most.
//
// A CTA has eight warps.  `wk` of them share its part of K, the others have 16 rows each of their own; the sums of those
// that share K are joined through shared memory in warp order.  CTAs are persistent; a warp's loads run on into
// its next rows while these are joined.  The tokens' values lie in shared memory, all of the CTA's part of K.  Where there
// are few rows, or more of K than shared memory holds, a cluster of CTAs shares K and each adds its share of the
// sums through distributed shared memory, in rank order.  Nothing depends on timing, and nothing needs a workspace.
//
// Measured (BF16, groups of 128): 1 x 6144 x 6144 8.7 us, of which the bytes would take 2.9 and launch, staging and joins
// take 4 to 5; 1 x 16384 x 8192 17.6 us (4.0 TB/s); 8 tokens 23.5 us, 16 tokens 31.5 us (groups of 64: 35.7).  At 16 tokens a step of
// 16 rows is some 220 warp instructions, which take less than half of the issue slots; the rest is waiting, for the tokens to be
// staged before the first product, for codes, and at the clusters' joins.  From 17 tokens on w4_tc.cu is faster (its figures
// are there).
// Before: weights made into whole FP16 numbers first, 13.4 us at 1 x 6144 x 6144; loads behind a branch, 22 us at 1 x 16384 x
// 8192; clusters counted as if all 76 of four CTAs fitted, 50 us at 16 tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ptx.cuh"
#include "w4.cuh"

namespace g13 {
namespace {

constexpr int WW = 8;            // warps of a CTA
constexpr int WT = WW * 32;
// CTAs per SM that the registers are kept for, and steps ahead of each warp.  (Of one to four CTAs and two to six steps,
// these were the fastest, or within 3 % of it, from 1 x 6144 x 6144 to 64 x 16384 x 8192.)
constexpr int w4_ctas(int nt) { return nt == 1 ? 3 : nt <= 4 ? 2 : 1; }
constexpr int w4_depth(int nt, int ng) { return nt == 1 && ng == 4 ? 2 : nt <= 2 ? 3 : 4; }

// Two 16-bit numbers to FP32.
__device__ __forceinline__ float2 two(uint32_t v, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// c = (or c +=) a 16 x 16 tile of weights times 16 values of 8 tokens.
template <bool FRESH>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (FRESH)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A code from the lowest place to the second lowest, in both halves of a register: by an integer multiplication (the mask
// comes after it), or of masked codes as FP16 numbers.  Either keeps off the pipe of the masks and shifts; one of
// each is the fastest (1 x 16384 x 8192: 17.6 us, shifts 18.9, FP16 alone 17.9).
__device__ __forceinline__ uint32_t up_int(uint32_t v) {
    uint32_t r;
    asm("mad.lo.u32 %0, %1, 16, 0;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t up_f16(uint32_t v) {
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v) : "r"(0x4C004C00u));
    return v;
}

// A step is 128 columns of 16 rows, two blocks.  As it is loaded: the codes, and of each of the NG groups that it
// meets the scales of rows g and g + 8 (two 16-bit numbers) and their zeros (two bytes).
template <int NG>
struct Step {
    uint4 lo, hi;
    uint32_t s[NG], z[NG];
};

// Shared memory: the tokens' rows (FP16); for each step, group and pair of tokens two sums and two powers of two; the
// warps' sums.  A token's row is 64 bytes longer than its values (a multiple of 256), so that the eight rows of a
// fragment load meet all banks.
__host__ __device__ constexpr int w4_row(int steps) { return steps * 256 + 64; }
// The sums of a token, from one to the next (the four extra spread the lanes' writes over the banks).
__host__ __device__ constexpr int w4_sum_row(int rows) { return rows + 4; }
struct W4Plan {
    int steps_rank;      // steps of K that a CTA has
    uint32_t inv_steps;  // its reciprocal (exact below 2^16; 0: one step)
    int windows;         // windows of a unit: DEPTH steps of each warp (some may not exist)
    uint32_t inv;        // reciprocal of group / 32 (exact below 2^16; 0: a group of 32)
    int blocks, tiles, groups, units;  // a unit: 16 rows to each of the 8 / WK warps that share no K
    int xvec;            // X takes 16-byte loads
    int bf16;
};
// WK warps share a CTA's part of K.  DENSE: a group is 128 / NG columns, so that groups follow one another as the
// steps do; else each step looks up its own.
template <int NT, int WK, int NG, bool DENSE, int DEPTH>
__global__ void __launch_bounds__(WT, w4_ctas(NT)) w4_kernel(const __grid_constant__ W4Args a, const __grid_constant__ W4Plan plan) {
    constexpr int TOK = 8 * NT, WR = WW / WK, ROWS = WR * 16;
    extern __shared__ __align__(128) uint8_t w4_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    uint32_t ranks, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int my_k = warp % WK, my_row = warp / WK;
    const int blocks = plan.blocks, tiles = plan.tiles, groups = plan.groups, steps_rank = plan.steps_rank;
    const bool bf16 = plan.bf16 != 0;  // of X and the scales
    const int first_block = min(static_cast<int>(rank) * steps_rank * 2, blocks);
    const int my_blocks = min(blocks - first_block, steps_rank * 2);
    const int my_steps = (my_blocks + 1) / 2;
    const int tok0 = static_cast<int>(blockIdx.y) * TOK, tok = min(TOK, static_cast<int>(a.M) - tok0);
    const int first = static_cast<int>(ranks == 1 ? blockIdx.x : blockIdx.x / ranks);
    const int stride = static_cast<int>(ranks == 1 ? gridDim.x : gridDim.x / ranks);
    const int row_bytes = w4_row(steps_rank);

    // ---- this warp's stream of steps, a window of DEPTH ahead
    Step<NG> ring[DEPTH] = {};
    int lj = my_k, ltile = first * WR + my_row;  // first step and tile of the next window that is loaded
    const int64_t tile_bytes = static_cast<int64_t>(blocks) * 512;
    const uint8_t* codes = a.codes + ltile * tile_bytes + static_cast<int64_t>(first_block + my_k * 2) * 512 + lane * 16;
    const int64_t entry = static_cast<int64_t>(ltile) * groups * 8 + g + (DENSE ? (first_block / 2 + my_k) * NG * 8 : 0);
    const uint32_t* scales = static_cast<const uint32_t*>(a.scales) + entry;
    // (without zeros: two eights, always the same ones)
    const uint16_t* zeros = a.zeros ? reinterpret_cast<const uint16_t*>(a.zeros) + entry : &kEights;
    const int zero_step = a.zeros ? 8 : 0;
    const auto load = [&](Step<NG>& b, int d) {
        const int j = lj + d * WK;
        const bool on = j < my_steps && ltile < tiles;
        const uint8_t* p = codes + d * (WK * 1024);
        ld_codes(b.lo, p, on);
        // (past the row's end any codes will do: the tokens' values there are zeros)
        ld_codes(b.hi, p + 512, on && 2 * j + 1 < my_blocks);
#pragma unroll
        for (int h = 0; h < NG; ++h) {
            int c = d * WK * NG + h;
            if (DENSE) {
                // (past the last group the last one again)
                if (NG > 1 && h > 0) c = d * WK * NG + min(h, groups - 1 - (first_block / 2 + j) * NG);
            } else {
                // the group of these columns: their place in units of 32 columns over group / 32
                c = min(over(static_cast<uint32_t>(first_block * 2 + j * 4 + h * (4 / NG)), plan.inv), groups - 1);
            }
            ld_nc32(b.s[h], scales + c * 8, on);
            ld_nc16(b.z[h], zeros + c * zero_step, on);
        }
    };
    const auto advance = [&] {
        lj += DEPTH * WK;
        codes += DEPTH * WK * 1024;
        if (DENSE) {
            scales += DEPTH * WK * NG * 8;
            zeros += DEPTH * WK * NG * zero_step;
        }
        if (lj >= plan.windows * DEPTH * WK) {  // the next unit
            const int back = plan.windows * DEPTH * WK;
            lj -= back;
            ltile += stride * WR;
            codes += stride * WR * tile_bytes - static_cast<int64_t>(back) * 1024;
            const int64_t on = static_cast<int64_t>(stride * WR) * groups - (DENSE ? back * NG : 0);
            scales += on * 8;
            zeros += on * zero_step;
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(ring[i], i);
    advance();

    // ---- the tokens' values of this CTA's part of K (zeros past the end).  Eight lanes take a step of a token, each
    // the 32 bytes that it asked for itself.
    float* pairs = reinterpret_cast<float*>(w4_raw + tok * row_bytes);  // [step][group][pair of tokens][4]
    float* sums = pairs + steps_rank * NG * TOK * 2;                    // [set][warp of K][token][row]
    {
        const int items = tok * steps_rank, piece = threadIdx.x & 7;
        const uint16_t* x = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(tok0) * a.ldx;
        const int k0 = first_block * 64 + piece * 16;
#pragma unroll 4
        for (int i = threadIdx.x >> 3; i < items; i += WT / 8) {
            const int t = over(i, plan.inv_steps), j = i - t * steps_rank, k = k0 + j * 128;
            const uint16_t* p = x + t * a.ldx + k;
            uint8_t* to = w4_raw + t * row_bytes + j * 256 + piece * 32;
            const int left = static_cast<int>(a.K) - k;  // (zeros behind the values that exist)
            if (plan.xvec) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = left - 8 * h;
                    cp_async_16z(smem_u32(to + 16 * h), n > 0 ? p + 8 * h : x, n >= 8 ? 16u : n > 0 ? static_cast<uint32_t>(n) * 2u : 0u);
                }
            } else {
                // aligned words, each of which holds at least one of the values, shifted
                const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1 & 1);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(p - odd);
                uint32_t e[9], v[8];
#pragma unroll
                for (int l = 0; l < 9; ++l) e[l] = 2 * l - odd < left && (l < 8 || odd) ? __ldg(q + l) : 0u;
#pragma unroll
                for (int l = 0; l < 8; ++l) {
                    v[l] = __funnelshift_r(e[l], e[l + 1], odd * 16);
                    if (2 * l + 1 >= left) v[l] = 2 * l >= left ? 0u : v[l] & 0xFFFFu;
                }
                reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        const unsigned lanes = 0xFFu << (lane & 24);
        for (int i = threadIdx.x >> 3; i < items; i += WT / 8) {
            const int t = over(i, plan.inv_steps), j = i - t * steps_rank;
            uint4* p = reinterpret_cast<uint4*>(w4_raw + t * row_bytes + j * 256 + piece * 32);
            const uint4 lo = p[0], hi = p[1];
            uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            float f[16], top = 0.0f, sum = 0.0f;
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const float2 h = two(w[l], bf16);
                f[2 * l] = h.x;
                f[2 * l + 1] = h.y;
            }
#pragma unroll
            for (int l = 0; l < 16; ++l) {
                top = fmaxf(top, fabsf(f[l]));  // (a NaN does not count)
                sum = fmaf(f[l], 0x1p-8f, sum);  // (the plain sum of 128 columns may lie beyond FP32)
            }
            if (top == INFINITY) {  // nor does an infinity
                top = 0.0f;
#pragma unroll
                for (int l = 0; l < 16; ++l) top = fabsf(f[l]) < INFINITY ? fmaxf(top, fabsf(f[l])) : top;
            }
            // the largest magnitude of the step, and from its exponent E the powers 2^(14 - E) and 2^(E - 6) (a group's
            // sum of 128 values below 2^15 and codes up to 15, times 2^-20, is below 2^6)
#pragma unroll
            for (int o = 1; o < 8; o *= 2) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
            const uint32_t biased = max(__float_as_uint(top) >> 23, 28u);  // (2^(14 - E) stays a normal number)
            const float up = __uint_as_float((127u + 14u + 127u - biased) << 23), down = __uint_as_float((biased - 6u) << 23);
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const __half2 h = __floats2half2_rn(f[2 * l] * up, f[2 * l + 1] * up);
                w[l] = *reinterpret_cast<const uint32_t*>(&h);
            }
            p[0] = make_uint4(w[0], w[2], w[1], w[3]);  // (two pairs for each of the two products)
            p[1] = make_uint4(w[4], w[6], w[5], w[7]);
#pragma unroll
            for (int o = 1; o < 8 / NG; o *= 2) sum += __shfl_xor_sync(lanes, sum, o);
            if (piece % (8 / NG) == 0) {  // (times 2^-20, like the products)
                float* q = pairs + ((j * NG + piece / (8 / NG)) * (TOK / 2) + t / 2) * 4 + t % 2;
                q[0] = sum * (up * 0x1p-12f);
                q[2] = down;
            }
        }
    }
    __syncthreads();

    float acc[NT][4];
    const auto clear = [&] {
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) acc[i / 4][i % 4] = 0.0f;
    };
    clear();
    // (columns past the last token read its values, and any sums: what comes of them is not used)
    const uint8_t* xrow[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xrow[n] = w4_raw + min(n * 8 + g, tok - 1) * row_bytes + my_k * 256 + t4 * 16;
    const float* xs = pairs + (my_k * NG * (TOK / 2) + t4) * 4;
    int j0 = 0;  // the window's first step, of the first warp of K
    const auto compute = [&](const Step<NG>& b, int d) {
        if (j0 + d * WK + my_k >= my_steps) return;
        float d0[NT][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            // 32 columns: sixteen bytes of each token, columns 32 h + 8 t4 .. + 7 of the step
            const uint4 v = h < 2 ? b.lo : b.hi;
            const uint32_t w0 = h & 1 ? v.z : v.x, w1 = h & 1 ? v.w : v.y, u0 = w0 >> 8, u1 = w1 >> 8;
            constexpr uint32_t LOW = 0x000F000Fu, AT = 0x00F000F0u;
            const uint32_t p0 = up_int(w0) & AT, p1 = up_int(w1) & AT, p2 = up_f16(u0 & LOW), p3 = up_f16(u1 & LOW);
            constexpr int LEN = 4 / NG;  // such pieces of a group
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x = *reinterpret_cast<const uint4*>(xrow[n] + j0 * 256 + d * (WK * 256) + h * 64);
                if (h % LEN == 0)
                    mma<true>(d0[n], p0, p1, p2, p3, x.x, x.y);
                else
                    mma<false>(d0[n], p0, p1, p2, p3, x.x, x.y);
                mma<false>(d0[n], w0 & AT, w1 & AT, u0 & AT, u1 & AT, x.z, x.w);
            }
            if ((h + 1) % LEN == 0) {
                const int gr = h / LEN;
                const float2 s = two(b.s[gr], bf16);
                // a zero as the lowest bits of 2^23
                const float z0 = __uint_as_float(__byte_perm(b.z[gr], 0x4B000000u, 0x7440)) - 0x1p23f;
                const float z1 = __uint_as_float(__byte_perm(b.z[gr], 0x4B000000u, 0x7441)) - 0x1p23f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 m = *reinterpret_cast<const float4*>(xs + j0 * (NG * TOK * 2) +
                                                                      (d * WK * NG + gr) * (TOK * 2) + n * 16);
                    const float e[4] = {fmaf(-z0, m.x, d0[n][0]), fmaf(-z0, m.y, d0[n][1]), fmaf(-z1, m.x, d0[n][2]),
                                        fmaf(-z1, m.y, d0[n][3])};
                    // (times the power first, which leaves the sum below FP32's largest; the power and a scale of
                    // another group of the step may not have a product)
                    acc[n][0] = fmaf(s.x, e[0] * m.z, acc[n][0]);
                    acc[n][1] = fmaf(s.x, e[1] * m.w, acc[n][1]);
                    acc[n][2] = fmaf(s.y, e[2] * m.z, acc[n][2]);
                    acc[n][3] = fmaf(s.y, e[3] * m.w, acc[n][3]);
                }
            }
        }
    };
    // The sums of a unit's rows: each CTA of the cluster adds its share of them, four rows of a token at a time, warps
    // and CTAs in order.  There are two sets of them in turn: one that is written is no longer read, since whoever
    // reads it has to arrive at the barrier of the unit in between.
    constexpr int SUM_ROW = w4_sum_row(ROWS);
    const int part = tok * SUM_ROW;
    int set = 0;
    const auto join = [&](int u) {
        float* base = sums + set * (WK * part);
        set ^= 1;
        float* mine = base + my_k * part + my_row * 16 + g;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int t = n * 8 + t4 * 2 + c;
                if (t >= tok) continue;
                // (2^20, of which the powers of two hold 2^8)
                mine[t * SUM_ROW] = acc[n][c] * 0x1p12f;
                mine[t * SUM_ROW + 8] = acc[n][2 + c] * 0x1p12f;
            }
        if (ranks > 1)
            cluster_sync();
        else
            __syncthreads();
        clear();
        const int count = tok * (ROWS / 4), step = WT * static_cast<int>(ranks);
        for (int i = static_cast<int>(rank) * WT + threadIdx.x; i < count; i += step) {
            const int t = i / (ROWS / 4), row = i % (ROWS / 4) * 4;
            const float* p = base + t * SUM_ROW + row;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const auto add = [&](const float4& o) {
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            };
            if (ranks == 1) {
#pragma unroll
                for (int w = 0; w < WK; ++w) add(*reinterpret_cast<const float4*>(p + w * part));
            } else {
                // (all loads of a warp of K are asked for before the first is used)
#pragma unroll 1
                for (int w = 0; w < WK; ++w) {
                    float4 o[8];
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k)
                        o[k] = k < ranks ? ld_cluster_f4(mapa_shared(smem_u32(p + w * part), k)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) add(o[k]);
                }
            }
            w4_store4(a.e, tok0 + t, static_cast<int64_t>(u) * ROWS + row, v);
        }
    };
    for (int u = first; u < plan.units; u += stride) {
        for (int w = 0; w < plan.windows; ++w) {
            j0 = w * (DEPTH * WK);
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                compute(ring[d], d);
                load(ring[d], d);
            }
            advance();
        }
        join(u);
    }
    if (ranks > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

int64_t w4_smem(int nt, int ng, int64_t tokens, int64_t steps_rank, int wk) {
    const int64_t tok = std::min<int64_t>(tokens, 8 * nt);
    return tok * w4_row(static_cast<int>(steps_rank)) + steps_rank * ng * 8 * nt * 8 +
           2 * wk * tok * w4_sum_row(WW / wk * 16) * 4;
}
// CTAs that an SM holds: by the registers that the kernel is compiled for, and its 228 KB (1 KB to each CTA itself).
int w4_per_sm(int nt, int64_t smem) { return static_cast<int>(std::min<int64_t>(w4_ctas(nt), 228 * 1024 / (smem + 1024))); }

template <int NT, int WK, int NG, bool DENSE>
cudaError_t launch(const W4Args& a, const W4Config& c, int num_sms, cudaStream_t st) {
    constexpr int DEPTH = w4_depth(NT, NG);
    auto k = w4_kernel<NT, WK, NG, DENSE, DEPTH>;
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Smem);
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    const int64_t steps = (a.K + 127) / 128;
    W4Plan p{};
    p.steps_rank = static_cast<int>((steps + c.splits - 1) / c.splits);
    p.inv_steps = reciprocal(p.steps_rank);
    p.windows = (p.steps_rank + DEPTH * WK - 1) / (DEPTH * WK);
    p.inv = reciprocal(a.group / 32);
    p.blocks = static_cast<int>(w4_blocks(a.K));
    p.tiles = static_cast<int>(w4_tiles(a.N));
    p.groups = static_cast<int>(w4_groups(a.K, a.group));
    p.xvec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.M <= 1 || a.ldx % 8 == 0);
    p.bf16 = a.dtype == GEMM_BF16;
    const int64_t smem = w4_smem(NT, NG, a.M, p.steps_rank, WK);
    const int64_t unit_rows = WW / WK * 16, units = (a.N + unit_rows - 1) / unit_rows;
    p.units = static_cast<int>(units);
    const int64_t at_once = std::max<int64_t>(1, std::max(1, w4_per_sm(NT, smem)) * clusters_at_once(c.splits, num_sms));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(units, at_once) * c.splits),
                       static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)));
    cfg.blockDim = dim3(WT);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (c.splits > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(c.splits);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, a, p);
}

template <int NG, bool DENSE>
cudaError_t launch_nt(const W4Config& c, const W4Args& a, int num_sms, cudaStream_t st) {
    switch (c.nt) {
        case 1: return c.wk == 8 ? launch<1, 8, NG, DENSE>(a, c, num_sms, st) : launch<1, 2, NG, DENSE>(a, c, num_sms, st);
        case 2: return launch<2, 2, NG, DENSE>(a, c, num_sms, st);
        case 4: return launch<4, 2, NG, DENSE>(a, c, num_sms, st);
        default: return launch<8, 2, NG, DENSE>(a, c, num_sms, st);
    }
}

// ------------------------------------------------------------------ to and from the layout
constexpr int CT = 256;

template <typename T>
__device__ __forceinline__ float f32(T v);
template <>
__device__ __forceinline__ float f32(float v) { return v; }
template <>
__device__ __forceinline__ float f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T cast(float v);
template <>
__device__ __forceinline__ float cast(float v) { return v; }
template <>
__device__ __forceinline__ __half cast(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 cast(float v) { return __float2bfloat16_rn(v); }

// Scale and zero of each group: a warp to one of them; rows past N: zeros.
template <typename T, typename S>
__global__ void __launch_bounds__(CT) w4_scales_kernel(const T* src, int64_t N, int64_t K, int64_t group, int64_t ld,
                                                       int64_t groups, S* scales, uint8_t* zeros) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (CT / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= w4_tiles(N) * 16 * groups) return;
    const int64_t r = i / groups, c = i - r * groups;
    float lo = 0.0f, hi = 0.0f;
    bool bad = false;
    if (r < N)
        for (int64_t k = c * group + lane; k < min(K, (c + 1) * group); k += 32) {
            const float v = f32(src[r * ld + k]);
            bad = bad || !(fabsf(v) < INFINITY);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane != 0) return;
    const float step = zeros ? hi * (1.0f / 15.0f) - lo * (1.0f / 15.0f) : fmaxf(hi, -lo) * (1.0f / 7.5f);
    const S s = cast<S>(bad ? __int_as_float(0x7FFFFFFF) : step);
    scales[w4_entry(r, c, groups)] = s;
    if (zeros) {
        const float d = f32(s);
        zeros[w4_entry(r, c, groups)] =
            static_cast<uint8_t>(d > 0.0f && d < INFINITY ? fminf(fmaxf(rintf(__fdiv_rn(-lo, d)), 0.0f), 15.0f) : 0.0f);
    }
}

// A thread to a word (eight codes); code(r, k): the code of an element that exists.
template <typename F>
__device__ __forceinline__ void write_word(int64_t N, int64_t K, uint32_t* codes, const F& code) {
    const int64_t words = w4_blocks(K) * 8, i = static_cast<int64_t>(blockIdx.x) * CT + threadIdx.x;
    const int64_t r = i / words, k = (i - r * words) * 8;
    if (r >= w4_tiles(N) * 16) return;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (r < N && k + j < K) w |= (code(r, k + j) & 15u) << (4 * (j % 2 * 4 + j / 2));
    codes[w4_word(r, k, w4_blocks(K))] = w;
}
template <typename T, typename S>
__global__ void __launch_bounds__(CT) w4_codes_kernel(const T* src, int64_t N, int64_t K, int64_t group, int64_t ld,
                                                      int64_t groups, uint32_t* codes, const S* scales,
                                                      const uint8_t* zeros) {
    write_word(N, K, codes, [&](int64_t r, int64_t k) {
        const int64_t e = w4_entry(r, k / group, groups);
        const float d = f32(scales[e]), z = zeros ? static_cast<float>(zeros[e]) : 8.0f;
        const float q = d > 0.0f ? __fdiv_rn(f32(src[r * ld + k]), d) : 0.0f;
        return static_cast<uint32_t>(fminf(fmaxf(rintf(q) + z, 0.0f), 15.0f));
    });
}
__global__ void __launch_bounds__(CT) w4_pack_codes_kernel(const uint8_t* q, int64_t N, int64_t K, int64_t ld,
                                                           uint32_t* codes) {
    write_word(N, K, codes, [&](int64_t r, int64_t k) { return static_cast<uint32_t>(q[r * ld + k]); });
}
__global__ void __launch_bounds__(CT) w4_pack_scales_kernel(const uint16_t* s, int64_t lds, const uint8_t* z,
                                                            int64_t ldz, int64_t N, int64_t groups, uint16_t* scales,
                                                            uint8_t* zeros) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * CT + threadIdx.x;
    const int64_t r = i / groups, c = i - r * groups;
    if (r >= w4_tiles(N) * 16) return;
    const int64_t e = w4_entry(r, c, groups);
    scales[e] = r < N ? s[r * lds + c] : uint16_t(0);
    if (zeros) zeros[e] = r < N ? z[r * ldz + c] & 15 : 0;
}
template <typename T, typename S>
__global__ void __launch_bounds__(CT) w4_dequantize_kernel(const uint32_t* codes, const S* scales, const uint8_t* zeros,
                                                           int64_t N, int64_t K, int64_t group, T* dst, int64_t ld) {
    const int64_t words = (K + 7) / 8, i = static_cast<int64_t>(blockIdx.x) * CT + threadIdx.x;
    const int64_t r = i / words, k = (i - r * words) * 8;
    if (r >= N) return;
    const uint32_t w = codes[w4_word(r, k, w4_blocks(K))];
    const int64_t e = w4_entry(r, k / group, w4_groups(K, group));  // (eight columns lie in one group)
    const float s = f32(scales[e]);
    const int z = zeros ? zeros[e] : 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < K)
            dst[r * ld + k + j] = cast<T>(static_cast<float>(static_cast<int>(w >> (4 * (j % 2 * 4 + j / 2)) & 15u) - z) * s);
}

unsigned grid_of(int64_t items, int per) { return static_cast<unsigned>((items + per - 1) / per); }

// f(T{}, S{}) with the types of `dtype` and of the 16-bit scales.
template <typename F>
cudaError_t with_types(int dtype, int scale_dtype, const F& f) {
    const auto s = [&](auto t) { return scale_dtype == GEMM_F16 ? f(t, __half()) : f(t, __nv_bfloat16()); };
    return dtype == GEMM_F32 ? s(float()) : dtype == GEMM_F16 ? s(__half()) : s(__nv_bfloat16());
}

}  // namespace

// The fewest passes over the weights that shared memory allows, then the cheapest cut by a model in ns: a CTA's
// steps take their bytes at its share of 45 bytes per ns and SM, or half a microsecond a turn where that is more; a
// unit's join 300, or 1800 where a cluster shares K.
W4Config w4_choose(int64_t M, int64_t N, int64_t K, int64_t group, int num_sms) {
    const int64_t steps = (K + 127) / 128;
    const int ng = w4_per_step(group);
    for (int nt = M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8;; nt /= 2) {
        W4Config best{nt, 0, 0};
        double least = 0;
        for (int s = 1; s <= 8; s *= 2)
            for (int wk = nt == 1 ? 8 : 2; wk >= 2; wk /= 4) {
                const int64_t rank_steps = (steps + s - 1) / s, turns = (rank_steps + wk - 1) / wk;
                const int64_t smem = w4_smem(nt, ng, M, rank_steps, wk);
                if (smem > kW4Smem || (s > 1 && (s - 1) * rank_steps >= steps)) continue;
                const int64_t rows = WW / wk * 16, passes = (M + 8 * nt - 1) / (8 * nt);
                const int64_t units = (N + rows - 1) / rows * passes;
                const int per_sm = w4_per_sm(nt, smem);
                const int64_t at_once = std::max<int64_t>(1, per_sm * clusters_at_once(s, num_sms));
                const int64_t rounds = (units + at_once - 1) / at_once;
                const int64_t ctas_sm = std::min<int64_t>(per_sm, (units * s + num_sms - 1) / num_sms);
                const double bytes = double(turns) * WW * 1024 * ctas_sm / 45.0;
                const double t = rounds * (std::max(bytes, turns * 500.0) + (s > 1 ? 1800 : 300)) +
                                 std::min<int64_t>(M, 8 * nt) * rank_steps * 256 * ctas_sm / 60.0;
                if (best.splits == 0 || t < least) {
                    least = t;
                    best.splits = s;
                    best.wk = wk;
                }
            }
        if (best.splits > 0) return best;
        if (nt == 1) return W4Config{1, 8, 8};  // (not reached: K is at most 65536)
    }
}

cudaError_t launch_w4(const W4Config& c, const W4Args& a, int num_sms, cudaStream_t st) {
    switch (a.group) {
        case 32: return launch_nt<4, true>(c, a, num_sms, st);
        case 64: return launch_nt<2, true>(c, a, num_sms, st);
        case 128: return launch_nt<1, true>(c, a, num_sms, st);
    }
    switch (w4_per_step(a.group)) {
        case 1: return launch_nt<1, false>(c, a, num_sms, st);
        case 2: return launch_nt<2, false>(c, a, num_sms, st);
        default: return launch_nt<4, false>(c, a, num_sms, st);
    }
}

cudaError_t launch_w4_quantize(int dtype, int scale_dtype, int64_t N, int64_t K, int64_t group, const void* src,
                               int64_t ld, uint8_t* codes, void* scales, uint8_t* zeros, cudaStream_t st) {
    const int64_t groups = w4_groups(K, group), rows = w4_tiles(N) * 16;
    return with_types(dtype, scale_dtype, [&](auto t, auto s) {
        using T = decltype(t);
        using S = decltype(s);
        w4_scales_kernel<T, S><<<grid_of(rows * groups, CT / 32), CT, 0, st>>>(
            static_cast<const T*>(src), N, K, group, ld, groups, static_cast<S*>(scales), zeros);
        w4_codes_kernel<T, S><<<grid_of(rows * w4_blocks(K) * 8, CT), CT, 0, st>>>(
            static_cast<const T*>(src), N, K, group, ld, groups, reinterpret_cast<uint32_t*>(codes),
            static_cast<const S*>(scales), zeros);
        return cudaGetLastError();
    });
}

cudaError_t launch_w4_pack(int64_t N, int64_t K, int64_t group, const uint8_t* q, int64_t ldq, const void* s,
                           int64_t lds, const uint8_t* z, int64_t ldz, uint8_t* codes, void* scales, uint8_t* zeros,
                           cudaStream_t st) {
    const int64_t groups = w4_groups(K, group), rows = w4_tiles(N) * 16;
    w4_pack_codes_kernel<<<grid_of(rows * w4_blocks(K) * 8, CT), CT, 0, st>>>(q, N, K, ldq,
                                                                              reinterpret_cast<uint32_t*>(codes));
    w4_pack_scales_kernel<<<grid_of(rows * groups, CT), CT, 0, st>>>(static_cast<const uint16_t*>(s), lds, z, ldz, N,
                                                                     groups, static_cast<uint16_t*>(scales), zeros);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(int dtype, int scale_dtype, int64_t N, int64_t K, int64_t group,
                                 const uint8_t* codes, const void* scales, const uint8_t* zeros, void* dst,
                                 int64_t ld, cudaStream_t st) {
    return with_types(dtype, scale_dtype, [&](auto t, auto s) {
        using T = decltype(t);
        using S = decltype(s);
        w4_dequantize_kernel<T, S><<<grid_of(N * ((K + 7) / 8), CT), CT, 0, st>>>(
            reinterpret_cast<const uint32_t*>(codes), static_cast<const S*>(scales), zeros, N, K, group,
            static_cast<T*>(dst), ld);
        return cudaGetLastError();
    });
}

}  // namespace g13
