// w4.cu -- products of a few tokens with 4-bit weights and group scales:
//
//   Y = cast( act( alpha sum_k X[m,k] (q[n,k] - z[n,k/g]) s[n,k/g] + bias[n] ) + beta R[m,n] )
//
// The weights' bytes are the cost (half a byte a weight); every one is read once, by 16-byte loads
// of whole 512-byte blocks, several blocks ahead in registers.  A warp multiplies a block of 16 rows
// x 64 columns with 8 tokens by four mma.sync m16n8k16: the weights are the 16 rows, the tokens the columns.
// A code becomes a 16-bit float by its bits alone: 128 + q in BF16 (1024 + q in FP16) has q as its lowest
// bits; taking off 128 + z leaves q - z exactly.  The group's scale multiplies the FP32 sum of its products
// (32 or 64 columns at a time), so no weight is rounded.
//
// A CTA of eight warps takes 16 (or 32) rows at a time; the warps take the blocks of a row in turn, so that
// the CTA reads whole kilobytes that follow one another, and their sums are joined through shared memory in warp
// order.  CTAs are persistent; a warp's loads run on into the CTA's next rows while these are joined.  The
// tokens' values lie in shared memory, all of the CTA's part of K.  Where there are few rows, or more of K than
// shared memory holds, a cluster of CTAs shares K and its first CTA adds the others' sums through
// distributed shared memory, in rank order.  Nothing depends on timing, and nothing needs a workspace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "w4.h"

namespace g13 {
namespace {

constexpr int WW = 8;            // warps of a CTA
constexpr int WT = WW * 32;
constexpr int kMaxDevices = 64;
constexpr int kW4Smem = 200 * 1024;  // at most, of the 227 KB that a CTA can have

template <typename T>
struct Half;
template <>
struct Half<__half> {
    static constexpr uint32_t magic = 0x64006400u;  // 1024, twice
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ float2 two(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <>
struct Half<__nv_bfloat16> {
    static constexpr uint32_t magic = 0x43004300u;  // 128, twice
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        const __nv_bfloat162 r =
            __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ float2 two(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A block as it is loaded: the codes, and of each group that it holds the scales of rows g and g + 8 (two 16-bit
// numbers) and their zeros (two bytes).
template <int R, int GROUPS>
struct Block {
    uint4 w[R];
    uint32_t s[R][GROUPS];
    uint32_t z[R][GROUPS];
};

// Shared memory: the tokens' rows, then the warps' sums.  A row is 64 bytes longer than its values (a multiple of
// 128), so that the eight rows of a fragment load meet all banks.
__host__ __device__ constexpr int w4_row(int blocks) { return blocks * 128 + 64; }
template <int NT, int R>
constexpr int kSumRow = 16 * R + 4;  // (the four extra spread the lanes' writes over the banks)
template <int NT, int R>
constexpr int kSums = 8 * NT * kSumRow<NT, R>;

// HALVES: groups of 32 columns, two to a block; else a block lies in one group.
template <typename T, int NT, int R, bool HALVES, int DEPTH>
__global__ void __launch_bounds__(WT) w4_kernel(const __grid_constant__ W4Args a, int kb_rank, bool xvec, uint32_t inv_group) {
    constexpr int GROUPS = HALVES ? 2 : 1, TOK = 8 * NT;
    extern __shared__ __align__(128) uint8_t w4_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    uint32_t ranks, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int blocks = static_cast<int>(w4_blocks(a.K)), tiles = static_cast<int>(w4_tiles(a.N));
    const int groups = static_cast<int>(w4_groups(a.K, a.group));
    const int kb0 = min(static_cast<int>(rank) * kb_rank, blocks), kb1 = min(kb0 + kb_rank, blocks);
    const int tok0 = static_cast<int>(blockIdx.y) * TOK, tok = min(TOK, static_cast<int>(a.M) - tok0);
    const int units = (tiles + R - 1) / R;
    const int first = static_cast<int>(blockIdx.x / ranks), step = static_cast<int>(gridDim.x / ranks);
    const int n_units = first < units ? (units - first + step - 1) / step : 0;
    const int turns = (kb_rank + WW - 1) / WW;  // blocks of a row tile that a warp takes (some may not exist)
    const int row_bytes = w4_row(kb_rank);
    float* sums = reinterpret_cast<float*>(w4_raw + tok * row_bytes);  // [warp][token][row]

    // ---- this warp's stream of blocks, DEPTH ahead
    Block<R, GROUPS> ring[DEPTH];
    int lu = first, lt = 0;  // unit and turn of the next load
    const auto load = [&](Block<R, GROUPS>& b) {
        const int kb = kb0 + lt * WW + warp;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int tile = lu * R + r;
            const bool on = kb < kb1 && tile < tiles && lu < units;
            if (!on) continue;
            b.w[r] = ld_codes(a.codes + (static_cast<int64_t>(tile) * blocks + kb) * 512 + lane * 16);
#pragma unroll
            for (int h = 0; h < GROUPS; ++h) {
                // the group of these 32 columns: their index over group / 32, by the reciprocal (exact
                // below 2^16; 0: group 32)
                const uint32_t i = static_cast<uint32_t>(kb * 2 + h);
                const int c = HALVES && inv_group == 0 ? min(static_cast<int>(i), groups - 1)
                                                       : min(static_cast<int>(__umulhi(i, inv_group)), groups - 1);
                const int64_t at = (static_cast<int64_t>(tile) * groups + c) * 8 + g;
                b.s[r][h] = __ldg(static_cast<const uint32_t*>(a.scales) + at);
                b.z[r][h] = a.zeros ? __ldg(reinterpret_cast<const uint16_t*>(a.zeros) + at) : 0x0808u;
            }
        }
        if (++lt == turns) {
            lt = 0;
            lu += step;
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(ring[i]);

    // ---- the tokens' values of this CTA's part of K (zeros past the end)
    {
        const uint16_t* x = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(tok0) * a.ldx;
        const int per = kb_rank * 8, k0 = kb0 * 64;  // 16-byte pieces of a row
        for (int i = threadIdx.x; i < tok * per; i += WT) {
            const int t = i / per, c = i - t * per, k = k0 + c * 8;
            const uint16_t* p = x + t * a.ldx + k;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (xvec && k + 8 <= a.K) {
                v = __ldg(reinterpret_cast<const uint4*>(p));
            } else {
                uint16_t e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = k + j < a.K ? __ldg(p + j) : uint16_t(0);
                v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
            }
            *reinterpret_cast<uint4*>(w4_raw + t * row_bytes + c * 16) = v;
        }
    }
    __syncthreads();

    float acc[R][NT][4];
    const auto clear = [&] {
#pragma unroll
        for (int i = 0; i < R * NT * 4; ++i) acc[i / (NT * 4)][i / 4 % NT][i % 4] = 0.0f;
    };
    clear();
    int u = first, turn = 0;
    const auto compute = [&](const Block<R, GROUPS>& b) {
        const int j = turn * WW + warp;  // block within the CTA's part of K
        if (kb0 + j >= kb1) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // sixteen bytes of each token: columns 32 h + 8 t4 .. + 7 of the block
            uint4 xv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                xv[n] = n * 8 + g < tok ? *reinterpret_cast<const uint4*>(w4_raw + (n * 8 + g) * row_bytes + j * 128 +
                                                                          h * 64 + t4 * 16)
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                constexpr uint32_t magic = Half<T>::magic;
                const int gr = HALVES ? h : 0;
                // magic + z, twice, of rows g and g + 8
                const uint32_t z0 = __byte_perm(b.z[r][gr], magic, 0x5050), z1 = __byte_perm(b.z[r][gr], magic, 0x5151);
                const uint32_t w0 = h == 0 ? b.w[r].x : b.w[r].z, w1 = h == 0 ? b.w[r].y : b.w[r].w;
                uint32_t p[4], q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = Half<T>::sub(((w0 >> (4 * i)) & 0x000F000Fu) | magic, z0);
                    q[i] = Half<T>::sub(((w1 >> (4 * i)) & 0x000F000Fu) | magic, z1);
                }
                const float2 sc = Half<T>::two(b.s[r][gr]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    Half<T>::mma(d, p[0], q[0], p[1], q[1], xv[n].x, xv[n].y);
                    Half<T>::mma(d, p[2], q[2], p[3], q[3], xv[n].z, xv[n].w);
                    acc[r][n][0] = fmaf(sc.x, d[0], acc[r][n][0]);
                    acc[r][n][1] = fmaf(sc.x, d[1], acc[r][n][1]);
                    acc[r][n][2] = fmaf(sc.y, d[2], acc[r][n][2]);
                    acc[r][n][3] = fmaf(sc.y, d[3], acc[r][n][3]);
                }
            }
        }
    };
    // The sums of a unit's rows: warps in order, then the cluster's CTAs in order.
    const auto join = [&] {
        float* mine = sums + warp * kSums<NT, R>;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[(n * 8 + t4 * 2 + (i & 1)) * kSumRow<NT, R> + r * 16 + g + (i >> 1) * 8] = acc[r][n][i];
        __syncthreads();
        clear();
        const int count = tok * 16 * R;
        for (int i = threadIdx.x; i < count; i += WT) {
            const int t = i / (16 * R), row = i % (16 * R);
            float* p = sums + t * kSumRow<NT, R> + row;
            float v = p[0];
#pragma unroll
            for (int w = 1; w < WW; ++w) v += p[w * kSums<NT, R>];
            if (ranks == 1)
                epi_store1(a.e, 0, tok0 + t, static_cast<int64_t>(u) * 16 * R + row, v);
            else
                p[0] = v;
        }
        if (ranks > 1) {
            cluster_sync();
            if (rank == 0) {
                for (int i = threadIdx.x; i < count; i += WT) {
                    const int t = i / (16 * R), row = i % (16 * R);
                    const float* p = sums + t * kSumRow<NT, R> + row;
                    float v = p[0];
                    for (uint32_t k = 1; k < ranks; ++k) {
                        float o;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(mapa_shared(smem_u32(p), k)) : "memory");
                        v += o;
                    }
                    epi_store1(a.e, 0, tok0 + t, static_cast<int64_t>(u) * 16 * R + row, v);
                }
            }
            cluster_sync();  // (the sums are read before they are written again, or the CTA leaves)
        } else {
            __syncthreads();
        }
    };
    const int total = n_units * turns;
    for (int i = 0; i < total; i += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (i + d >= total) break;
            compute(ring[d]);
            load(ring[d]);
            if (++turn == turns) {
                join();
                turn = 0;
                u += step;
            }
        }
    }
}

template <typename T, int NT, int R, bool HALVES, int DEPTH>
cudaError_t launch(const W4Args& a, int splits, int num_sms, cudaStream_t st) {
    auto k = w4_kernel<T, NT, R, HALVES, DEPTH>;
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Smem);
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    const int kb_rank = static_cast<int>((w4_blocks(a.K) + splits - 1) / splits);
    const int tok = static_cast<int>(std::min<int64_t>(a.M, 8 * NT));
    const int smem = tok * w4_row(kb_rank) + WW * kSums<NT, R> * 4;
    const int64_t units = (w4_tiles(a.N) + R - 1) / R;
    int per_sm = 0;
    ce = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, WT, smem);
    if (ce != cudaSuccess) return ce;
    const int64_t at_once = std::max<int64_t>(1, static_cast<int64_t>(per_sm) * num_sms / splits);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(units, at_once) * splits),
                       static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)));
    cfg.blockDim = dim3(WT);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (splits > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(splits);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    const bool xvec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.M <= 1 || a.ldx % 8 == 0);
    const uint32_t per = static_cast<uint32_t>(a.group / 32);
    const uint32_t inv = per == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + per - 1) / per);
    return cudaLaunchKernelEx(&cfg, k, a, kb_rank, xvec, inv);
}

// Row tiles of a unit: two where a token's values would be read from shared memory faster than the weights come.
constexpr int w4_r(int nt) { return nt == 1 ? 1 : 2; }
template <int NT>
int64_t w4_smem(int64_t tokens, int64_t kb_rank) {
    return std::min<int64_t>(tokens, 8 * NT) * w4_row(static_cast<int>(kb_rank)) + WW * kSums<NT, w4_r(NT)> * 4;
}
int64_t w4_smem(int nt, int64_t tokens, int64_t kb_rank) {
    return nt == 1   ? w4_smem<1>(tokens, kb_rank)
           : nt == 2 ? w4_smem<2>(tokens, kb_rank)
           : nt == 4 ? w4_smem<4>(tokens, kb_rank)
                     : w4_smem<8>(tokens, kb_rank);
}

template <typename T, bool HALVES>
cudaError_t launch_nt(const W4Config& c, const W4Args& a, int num_sms, cudaStream_t st) {
    switch (c.nt) {
        case 1: return launch<T, 1, w4_r(1), HALVES, 4>(a, c.splits, num_sms, st);
        case 2: return launch<T, 2, w4_r(2), HALVES, 2>(a, c.splits, num_sms, st);
        case 4: return launch<T, 4, w4_r(4), HALVES, 2>(a, c.splits, num_sms, st);
        default: return launch<T, 8, w4_r(8), HALVES, 2>(a, c.splits, num_sms, st);
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

// The fewest passes over the weights that shared memory allows, then CTAs of a cluster to a row tile's K: as many
// as it takes for the tokens' values to fit, and more (up to 8, eight blocks of K each at least) while all row
// tiles leave SMs without work.
W4Config w4_choose(int64_t M, int64_t N, int64_t K, int num_sms) {
    const int64_t blocks = w4_blocks(K);
    for (int nt = M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8;; nt /= 2) {
        const int64_t units = (w4_tiles(N) + w4_r(nt) - 1) / w4_r(nt) * ((M + 8 * nt - 1) / (8 * nt));
        for (int s = 1; s <= 8; s *= 2) {
            if (w4_smem(nt, M, (blocks + s - 1) / s) > kW4Smem) continue;
            while (s < 8 && units * s * 2 <= num_sms * 2 && blocks >= 16 * s) s *= 2;
            return W4Config{nt, s};
        }
        if (nt == 1) return W4Config{1, 8};  // (not reached: K is at most 65536)
    }
}

cudaError_t launch_w4(const W4Config& c, const W4Args& a, int num_sms, cudaStream_t st) {
    const bool f16 = a.dtype == GEMM_F16, halves = a.group % 64 != 0;
    if (halves)
        return f16 ? launch_nt<__half, true>(c, a, num_sms, st) : launch_nt<__nv_bfloat16, true>(c, a, num_sms, st);
    return f16 ? launch_nt<__half, false>(c, a, num_sms, st) : launch_nt<__nv_bfloat16, false>(c, a, num_sms, st);
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
