// fp4_gemm.cu -- the product of two microscaled 4-bit matrices on the tensor
// cores:  C = cast(act(alpha gA gB sum_k a[m,k] b[n,k] + bias[n]) + beta R[m,n])
//
// tcgen05.mma kind::mxf4 / mxf4nvf4 multiplies E2M1 codes straight from
// shared memory and applies the block scales, read from TMEM, inside the
// instruction, accumulating in FP32; the tensor scales gA, gB go into the
// epilogue's factor.  64 K elements are one instruction (32 bytes of a
// 128-byte-swizzled row), so a ring stage holds K = 256: rows of 128 bytes.
//
// The rows of B (a weight's output columns) take the 128 TMEM lanes and the
// rows of A (tokens) the accumulator's columns, from 16 of them for decoding
// to 256: a few tokens then cost their own width only, while each weight row is
// streamed once at full tile height.  A warp's 32 lanes hold 32 neighbouring
// columns of a C row, so every store of the epilogue is one contiguous piece
// of a row at any alignment, with no transpose through shared memory, and the
// bias is one value per thread.
//
//   warp 0      producer: TMA boxes of both operands' codes and bulk copies of
//               their scale tiles into a ring, counted by full[s]
//   warp 1      one thread: tcgen05.cp of the stage's scale tiles to TMEM (in
//               order with the MMAs that read them), then the MMAs; commits
//               free ring stages (empty[s]) and finish accumulators (tfull)
//   warps 2..5  epilogue, one TMEM lane quarter each
//
// Few tokens leave fewer tiles than SMs: a cluster then splits K, each CTA
// leaves its partial sums in its own shared memory, and every CTA adds one
// share of the columns through distributed shared memory, in rank order (the
// result does not depend on timing, and needs no workspace).
//
// Every wait is bounded; after a timeout the CTA lets its own copies and MMAs
// land, frees TMEM and leaves, and the plan's status word records it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "fp4_gemm.h"
#include "tc_kernel.cuh"

namespace g13 {
namespace {

constexpr int FW = 128;            // weight rows (TMEM lanes) of a tile
constexpr int F_KB = 256;          // K elements per stage: 128 bytes of codes
constexpr int F_W_TILE = FW * 128;
constexpr int F_THREADS = 192;

template <int BN, int FMT>
struct F4Layout {
    static constexpr int CT = F_KB / (4 * fp4_block(FMT));  // scale tiles per stage along K
    static constexpr int XT = (BN + 127) / 128;             // row tiles of the token side
    static constexpr int X_TILE = BN * 128;
    static constexpr int SFW_BYTES = CT * kFp4TileBytes;
    static constexpr int SFX_BYTES = XT * CT * kFp4TileBytes;
    static constexpr int STAGE_BYTES = F_W_TILE + X_TILE + SFW_BYTES + SFX_BYTES;
    static constexpr int STAGE_ALIGN = (STAGE_BYTES + 1023) / 1024 * 1024;
    // accumulators, then two sets of scale columns (a tile is 4 columns)
    static constexpr int NBUF = BN > 128 ? 1 : 2;
    static constexpr int SF_COLS = CT * 4 * (1 + XT);
    static constexpr int SF_BASE = NBUF * BN;
    static constexpr int COLS = SF_BASE + 2 * SF_COLS;
    static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
};

struct F4Args {
    int64_t M, N, K;
    const uint8_t* sw;  // scale tiles of the weight side (B) and of the tokens (A)
    const uint8_t* sx;
    const float* gw;    // tensor scales, or null
    const float* gx;
    int64_t w_tiles, x_tiles;    // row tiles of 128 that exist on each side
    int64_t n_tiles, m_tiles;    // tiles of the product
    int col_tiles;               // scale tiles along K
    int k_blocks;                // stages along K
    int raster;
    uint32_t idesc;
    EpiParams e;
    unsigned* status;
    uint64_t timeout_ns;
    uint32_t flags;
};

// No-swizzle descriptor of one scale tile for tcgen05.cp: 32 rows of 16 bytes,
// groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    uint64_t d = (saddr >> 4) & 0x3FFFu;
    d |= static_cast<uint64_t>(128 >> 4) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}
// One scale tile (512 bytes) into four TMEM columns of all four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
    if (FMT == GEMM_MXFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
}
// Untiled bulk copy into shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}
// 16 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// alpha' acc + bias -> act -> + beta R -> cast of CN columns of C rows m0..: one element per lane and row.
template <int CN>
__device__ __forceinline__ void f4_store(const EpiParams& e, float alpha, float bias, int64_t m0,
                                         int64_t n, float* v) {
    if (n >= e.N) return;
    const int live = static_cast<int>(min(static_cast<int64_t>(CN), e.M - m0));
    float r[CN];
    if (e.R) {
#pragma unroll
        for (int j = 0; j < CN; ++j)
            r[j] = j < live ? __ldg(e.R + (m0 + j) * e.ldr + n) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < CN; ++j) v[j] = fmaf(v[j], alpha, bias);
    if (e.act == GEMM_ACT_GELU_ERF) {
#pragma unroll
        for (int j = 0; j < CN; j += 2) gelu2_as7126(v[j], v[j + 1]);
    } else if (e.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < CN; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    }
    if (e.R) {
#pragma unroll
        for (int j = 0; j < CN; ++j) v[j] = fmaf(e.beta, r[j], v[j]);
    }
    if (e.out_dtype == GEMM_F32) {
        float* c = static_cast<float*>(e.C) + m0 * e.ldc + n;
#pragma unroll
        for (int j = 0; j < CN; ++j)
            if (j < live) c[j * e.ldc] = v[j];
    } else if (e.out_dtype == GEMM_BF16) {
        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(e.C) + m0 * e.ldc + n;
#pragma unroll
        for (int j = 0; j < CN; ++j)
            if (j < live) c[j * e.ldc] = __float2bfloat16_rn(v[j]);
    } else {
        __half* c = static_cast<__half*>(e.C) + m0 * e.ldc + n;
#pragma unroll
        for (int j = 0; j < CN; ++j)
            if (j < live) c[j * e.ldc] = __float2half_rn(v[j]);
    }
}

template <int BN, int STAGES, int FMT>
constexpr int f4_smem() {
    return 1024 + STAGES * F4Layout<BN, FMT>::STAGE_ALIGN + (2 * STAGES + 5) * 8 + 16;
}

__device__ __forceinline__ void f4_tile(const F4Args& a, int64_t t, int64_t& mt, int64_t& nt) {
    // groups of `raster` weight tiles, token tiles fastest within a group
    const uint32_t tu = static_cast<uint32_t>(t), m = static_cast<uint32_t>(a.m_tiles);
    const uint32_t span = static_cast<uint32_t>(a.raster) * m;
    const uint32_t g = tu / span, first = g * static_cast<uint32_t>(a.raster);
    const uint32_t gn = min(static_cast<uint32_t>(a.raster), static_cast<uint32_t>(a.n_tiles) - first);
    const uint32_t w = tu - g * span;
    nt = first + w % gn;
    mt = w / gn;
}

// SPLIT: one tile per cluster, K divided over its CTAs.  Else persistent, one CTA per tile at a time.
template <int BN, int STAGES, int FMT, bool SPLIT>
__global__ void __launch_bounds__(F_THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const F4Args args) {
    using L = F4Layout<BN, FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * L::STAGE_ALIGN);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&tfull[i]), 1);
            mbar_init(smem_u32(&tempty[i]), 128);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t tmo = args.timeout_ns;

    const uint32_t rank = SPLIT ? cluster_ctarank() : 0u;
    uint32_t splits = 1;
    if (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    const int64_t t_begin = SPLIT ? blockIdx.x / splits : blockIdx.x;
    const int64_t t_step = SPLIT ? args.n_tiles * args.m_tiles : gridDim.x;
    const int64_t t_end = args.n_tiles * args.m_tiles;
    const int kb_lo = SPLIT ? static_cast<int>(static_cast<int64_t>(args.k_blocks) * rank / splits) : 0;
    const int kb_hi = SPLIT ? static_cast<int>(static_cast<int64_t>(args.k_blocks) * (rank + 1) / splits)
                            : args.k_blocks;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ producer
            const bool stall = (args.flags & GEMM_FLAG_TEST_STALL) && blockIdx.x == 0;
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            bool ok = true;
            for (int64_t t = t_begin; ok && t < t_end; t += t_step) {
                int64_t mt, nt;
                f4_tile(args, t, mt, nt);
                const int64_t xt0 = mt * BN / 128;  // first row tile of the token side
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&empty[s]), ph ^ 1u, abort_flag, args.status, tmo)) {
                        ok = false;
                        break;
                    }
                    armed &= ~(1u << s);
                    if (!(stall && t == t_begin && kb == kb_lo)) {
                        const uint32_t st = smem_u32(smem + s * L::STAGE_ALIGN);
                        const uint32_t bar = smem_u32(&full[s]);
                        const int c0 = kb * L::CT;
                        const uint32_t sf = static_cast<uint32_t>(min(L::CT, args.col_tiles - c0)) * kFp4TileBytes;
                        const bool two = L::XT == 2 && xt0 + 1 < args.x_tiles;
                        mbar_arrive_expect_tx(bar, F_W_TILE + L::X_TILE + sf * (two ? 3 : 2));
                        tma_load_3d(st, &tmW, bar, kb * 128, static_cast<int32_t>(nt * FW), 0);
                        tma_load_3d(st + F_W_TILE, &tmX, bar, kb * 128, static_cast<int32_t>(mt * BN), 0);
                        const uint32_t dst = st + F_W_TILE + L::X_TILE;
                        bulk_load(dst, args.sw + (nt * args.col_tiles + c0) * kFp4TileBytes, sf, bar);
                        bulk_load(dst + L::SFW_BYTES, args.sx + (xt0 * args.col_tiles + c0) * kFp4TileBytes, sf,
                                  bar);
                        if (two)
                            bulk_load(dst + 2 * L::SFW_BYTES,
                                      args.sx + ((xt0 + 1) * args.col_tiles + c0) * kFp4TileBytes, sf, bar);
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    }
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok)
                for (int i = 0; i < STAGES; ++i)
                    if (armed & (1u << i)) tc_drain(smem_u32(&full[i]), (armed_par >> i) & 1u, tmo);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuer
            int s = 0, lt = 0;
            uint32_t ph = 0, set = 0;
            bool ok = true, issued = false;
            for (int64_t t = t_begin; ok && t < t_end; t += t_step, ++lt) {
                const int buf = L::NBUF == 1 ? 0 : (lt & 1);
                const uint32_t tph = static_cast<uint32_t>(L::NBUF == 1 ? lt : (lt >> 1)) & 1u;
                if (!mbar_wait_bounded(smem_u32(&tempty[buf]), tph ^ 1u, abort_flag, args.status, tmo)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&full[s]), ph, abort_flag, args.status, tmo)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * L::STAGE_ALIGN);
                    const uint32_t sfs = st + F_W_TILE + L::X_TILE;
                    const uint32_t sf_t = tmem_base + L::SF_BASE + (set ? L::SF_COLS : 0);
                    set ^= 1u;
                    const int ct = min(L::CT, args.col_tiles - kb * L::CT);
                    // TMEM columns of tile c: weights at 4c, tokens' row tile x at 4 (CT + c XT + x)
                    for (int c = 0; c < ct; ++c) {
                        sf_copy(sf_t + 4 * c, sf_desc(sfs + c * kFp4TileBytes));
#pragma unroll
                        for (int x = 0; x < L::XT; ++x)
                            sf_copy(sf_t + 4 * (L::CT + c * L::XT + x),
                                    sf_desc(sfs + L::SFW_BYTES * (1 + x) + c * kFp4TileBytes));
                    }
                    const int steps = static_cast<int>(min(static_cast<int64_t>(F_KB), args.K - static_cast<int64_t>(kb) * F_KB) + 63) / 64;
                    for (int kk = 0; kk < steps; ++kk) {
                        // nvfp4: a tile per step; mxfp4: two steps share a tile, bytes 0-1 and 2-3
                        const int c = FMT == GEMM_MXFP4 ? kk >> 1 : kk;
                        const uint32_t id = FMT == GEMM_MXFP4 ? (kk & 1) * 2u : 0u;
                        mma_f4<FMT>(d, smem_desc_sw128(st + kk * 32, 16, 1024),
                                    smem_desc_sw128(st + F_W_TILE + kk * 32, 16, 1024),
                                    args.idesc | (id << 29) | (id << 4), sf_t + 4 * c,
                                    sf_t + 4 * (L::CT + c * L::XT), (kb > kb_lo || kk > 0) ? 1u : 0u);
                    }
                    issued = true;
                    tc_commit(smem_u32(&empty[s]));
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(smem_u32(&tfull[buf]));
            }
            if (!ok && issued) {
                tc_commit(smem_u32(drain));
                tc_drain(smem_u32(drain), 0u, tmo);
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        float alpha = args.e.alpha;
        if (args.gw) alpha *= __ldg(args.gw);
        if (args.gx) alpha *= __ldg(args.gx);
        int lt = 0;
        for (int64_t t = t_begin; t < t_end; t += t_step, ++lt) {
            int64_t mt, nt;
            f4_tile(args, t, mt, nt);
            const int64_t n = nt * FW + q * 32 + lane;
            const float bias = args.e.bias && n < args.N ? __ldg(args.e.bias + n) : 0.0f;
            const int buf = L::NBUF == 1 ? 0 : (lt & 1);
            const uint32_t tph = static_cast<uint32_t>(L::NBUF == 1 ? lt : (lt >> 1)) & 1u;
            // the whole warp goes on or leaves: the TMEM loads are warp-wide
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(&tfull[buf]), tph, abort_flag,
                                                           args.status, tmo)))
                break;
            tc_fence_after();
            // K = 0 (or an empty share of K) issued no MMA: the sum is zero
            const bool none = kb_lo == kb_hi;
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                if (!SPLIT && mt * BN + c >= args.M) break;
                uint32_t r[16];
                tmem_ld_x16(tmem_base + lane_base + static_cast<uint32_t>(buf * BN + c), r);
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = none ? 0.0f : __uint_as_float(r[j]);
                if (SPLIT) {
                    // every MMA of this CTA is done: the ring is free for the partial sums [column][lane]
                    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * FW + q * 32 + lane] = v[j];
                } else {
                    f4_store<16>(args.e, alpha, bias, mt * BN + c, n, v);
                    __syncwarp();
                }
            }
            if (!SPLIT) {
                tc_fence_before();
                mbar_arrive(smem_u32(&tempty[buf]));
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= 2) {
            int64_t mt, nt;
            f4_tile(args, t_begin, mt, nt);
            const int q = warp & 3;
            const int64_t n = nt * FW + q * 32 + lane;
            float alpha = args.e.alpha;
            if (args.gw) alpha *= __ldg(args.gw);
            if (args.gx) alpha *= __ldg(args.gx);
            const float bias = args.e.bias && n < args.N ? __ldg(args.e.bias + n) : 0.0f;
            // a CTA that gave up leaves its sums undefined: nothing is written (the status says so)
            const int cols = static_cast<int>(min(static_cast<int64_t>(BN), args.M - mt * BN));
            const uint32_t part = smem_u32(smem) + (q * 32 + lane) * 4;
            // pairs of columns in turn over the ranks
            for (int c = 2 * static_cast<int>(rank); c < cols; c += 2 * static_cast<int>(splits)) {
                float v[2] = {0.0f, 0.0f};
                for (uint32_t p = 0; p < splits; ++p) {
                    const uint32_t src = mapa_shared(part + c * FW * 4, p);
                    v[0] += ld_cluster_f32(src);
                    v[1] += ld_cluster_f32(src + FW * 4);
                }
                f4_store<2>(args.e, alpha, bias, mt * BN + c, n, v);
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while others read its shared memory
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, L::TMEM_COLS);
}

template <int BN, int STAGES, int FMT, bool SPLIT>
cudaError_t launch_f4(const CUtensorMap& tmW, const CUtensorMap& tmX, const F4Args& a, int splits,
                      int num_sms, cudaStream_t st) {
    auto k = fp4_gemm_kernel<BN, STAGES, FMT, SPLIT>;
    constexpr int smem = f4_smem<BN, STAGES, FMT>();
    static_assert(smem <= kMaxDynSmem, "shared memory");
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    const int64_t tiles = a.n_tiles * a.m_tiles;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? tiles * splits : std::min<int64_t>(tiles, num_sms)));
    cfg.blockDim = dim3(F_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (SPLIT) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(splits);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, tmW, tmX, a);
}

template <int BN, int STAGES>
cudaError_t launch_fmt(int fmt, const CUtensorMap& tmW, const CUtensorMap& tmX, const F4Args& a, int splits,
                       int num_sms, cudaStream_t st) {
    if constexpr (BN <= 128) {
        if (splits > 1)
            return fmt == GEMM_MXFP4
                       ? launch_f4<BN, STAGES, GEMM_MXFP4, true>(tmW, tmX, a, splits, num_sms, st)
                       : launch_f4<BN, STAGES, GEMM_NVFP4, true>(tmW, tmX, a, splits, num_sms, st);
    }
    return fmt == GEMM_MXFP4 ? launch_f4<BN, STAGES, GEMM_MXFP4, false>(tmW, tmX, a, 1, num_sms, st)
                             : launch_f4<BN, STAGES, GEMM_NVFP4, false>(tmW, tmX, a, 1, num_sms, st);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Config& c, int fmt, const CUtensorMap& tmW, const CUtensorMap& tmX,
                            const uint8_t* sw, const float* gw, const uint8_t* sx, const float* gx, int64_t K,
                            const EpiParams& e, const LaunchCtx& lc) {
    F4Args a{};
    a.M = e.M;
    a.N = e.N;
    a.K = K;
    a.sw = sw;
    a.sx = sx;
    a.gw = gw;
    a.gx = gx;
    a.w_tiles = fp4_row_tiles(e.N);
    a.x_tiles = fp4_row_tiles(e.M);
    a.n_tiles = (e.N + FW - 1) / FW;
    a.m_tiles = (e.M + c.bn - 1) / c.bn;
    a.col_tiles = static_cast<int>(fp4_col_tiles(fmt, K));
    a.k_blocks = static_cast<int>((K + F_KB - 1) / F_KB);
    a.raster = 8;
    a.e = e;
    a.status = lc.status;
    a.timeout_ns = lc.timeout_ns;
    a.flags = lc.flags;
    // instruction descriptor: E2M1 operands (1), scale type (1: UE8M0), N, M = 128
    a.idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(c.bn >> 3) << 17) |
              ((fmt == GEMM_MXFP4 ? 1u : 0u) << 23) | (static_cast<uint32_t>(FW >> 7) << 27);
    switch (c.bn) {
        case 16: return launch_fmt<16, 8>(fmt, tmW, tmX, a, c.splits, lc.num_sms, lc.stream);
        case 32: return launch_fmt<32, 8>(fmt, tmW, tmX, a, c.splits, lc.num_sms, lc.stream);
        case 64: return launch_fmt<64, 7>(fmt, tmW, tmX, a, c.splits, lc.num_sms, lc.stream);
        case 128: return launch_fmt<128, 6>(fmt, tmW, tmX, a, c.splits, lc.num_sms, lc.stream);
        case 256: return launch_fmt<256, 4>(fmt, tmW, tmX, a, c.splits, lc.num_sms, lc.stream);
        default: return cudaErrorInvalidValue;
    }
}

// Tokens per tile: the narrowest of 16, 32, 64 that holds them all; above 64,
// 256-wide tiles once they fill the GPU, else 128.  K is split over a cluster
// while the tiles leave SMs idle.
Fp4Config fp4_choose(int64_t M, int64_t N, int64_t K, int num_sms) {
    Fp4Config c{};
    const int64_t n_tiles = (N + FW - 1) / FW;
    if (M <= 16)
        c.bn = 16;
    else if (M <= 32)
        c.bn = 32;
    else if (M <= 64)
        c.bn = 64;
    else
        c.bn = ((M + 255) / 256) * n_tiles >= num_sms ? 256 : 128;
    c.splits = 1;
    const int64_t tiles = n_tiles * ((M + c.bn - 1) / c.bn);
    const int64_t kbs = (K + F_KB - 1) / F_KB;
    if (c.bn <= 128 && tiles > 0 && kbs > 1) {
        const int64_t most = std::min<int64_t>(8, kbs);
        c.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, num_sms / tiles)));
    }
    return c;
}

}  // namespace g13
