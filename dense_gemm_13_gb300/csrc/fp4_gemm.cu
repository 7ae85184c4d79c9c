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
//   warp 0      producer: TMA boxes of both operands' codes and scale tiles into
//               a ring, counted by full[s]
//   warp 1      tcgen05.cp of the stage's scale tiles to TMEM (in order with the
//               MMAs that read them), then the MMAs, by one elected lane; commits
//               free ring stages (empty[s]) and finish accumulators (tfull)
//   others      epilogue: four warps, one TMEM lane quarter each, or 16, four to a
//               quarter, taking its 32-column chunks in turn
//
// Large products run on CTA pairs (tcgen05 cta_group::2): 256 weight rows x 256
// tokens, each CTA holding its own 128 weight rows and half of the tokens, so
// that a stage brings 38 KB into each SM instead of 54 KB for 128 x 256.  At
// 8192^3 (nvfp4) that is 185-190 us, 5.8-5.9 PFLOP/s: the tensor cores are busy 66 %
// of the cycles, and 14 TB/s come from L2, close to the 15 TB/s that the same loads
// reached with nothing else running.  256 accumulator columns and the scales do not fit TMEM twice: two
// accumulators overlap by 96 columns, which the epilogue reads first and hands
// back, so the next tile's MMAs start before the rest is stored.
//
// Up to 64 tokens the weights' bytes are the cost (1 x 6144 x 6144: 8.0 us, of
// which 3.2 would be HBM's share and 3 the launch, set-up and cluster barriers).
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
enum F4Mode { F4_ONE = 0, F4_SPLIT = 1, F4_PAIR = 2 };

template <int BN, int FMT, int MODE>
struct F4Layout {
    static constexpr bool PAIR = MODE == F4_PAIR;
    static constexpr int EW = BN >= 128 ? 16 : 4;           // epilogue warps
    static constexpr int THREADS = 64 + 32 * EW;
    static constexpr int TILE_W = PAIR ? 2 * FW : FW;       // weight rows of a tile
    static constexpr int X_ROWS = PAIR ? BN / 2 : BN;       // tokens that this CTA loads
    static constexpr int CT = F_KB / (4 * fp4_block(FMT));  // scale tiles per stage along K
    static constexpr int XT = (BN + 127) / 128;             // row tiles of the token side
    static constexpr int X_TILE = X_ROWS * 128;
    static constexpr int SFW_BYTES = CT * kFp4TileBytes;
    static constexpr int SFX_BYTES = XT * CT * kFp4TileBytes;
    static constexpr int STAGE_BYTES = F_W_TILE + X_TILE + SFW_BYTES + SFX_BYTES;
    static constexpr int STAGE_ALIGN = (STAGE_BYTES + 1023) / 1024 * 1024;
    // TMEM columns: two accumulators ACC_STEP apart (side by side, or overlapping
    // where BN = 256), then sets of scale columns (a tile is 4 columns), one per stage in
    // turn: up to one less than the ring's stages, or the two that 256 x 256 tiles leave room
    // for in nvfp4
    static constexpr int OVERLAP = BN == 256 ? 96 : 0;
    static constexpr int ACC_STEP = BN - OVERLAP;
    static constexpr int SF_COLS = CT * 4 * (1 + XT);
    static constexpr int SF_BASE = ACC_STEP + BN;
    static constexpr int SETS = BN <= 32 ? 7 : BN == 64 ? 6 : SF_BASE + 4 * SF_COLS <= 512 ? 4 : 2;
    static constexpr int COLS = SF_BASE + SETS * SF_COLS;
    static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(COLS <= 512, "TMEM");
};

struct F4Args {
    int64_t M, N, K;
    const float* gw;             // tensor scales of the weight side (B) and the tokens (A), or null
    const float* gx;
    int64_t n_tiles, m_tiles;    // tiles of the product
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
// One scale tile (512 bytes) into four TMEM columns of all four lane quarters
// (of both CTAs of a pair, each from its own shared memory).
template <bool PAIR>
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t sdesc) {
    if (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
#define G13_MMA_F4(group, kind, vec)                                                                    \
    asm volatile(                                                                                       \
        "{\n\t.reg .pred p;\n\t"                                                                        \
        "setp.ne.b32 p, %6, 0;\n\t"                                                                     \
        "tcgen05.mma.cta_group::" group ".kind::" kind ".block_scale.scale_vec::" vec                   \
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                              \
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                                        \
        : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
    if (FMT == GEMM_MXFP4) {
        if (PAIR)
            G13_MMA_F4("2", "mxf4", "2X");
        else
            G13_MMA_F4("1", "mxf4", "2X");
    } else {
        if (PAIR)
            G13_MMA_F4("2", "mxf4nvf4", "4X");
        else
            G13_MMA_F4("1", "mxf4nvf4", "4X");
    }
}
#undef G13_MMA_F4
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A bounded wait of a whole warp: the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                               unsigned* status, uint64_t timeout_ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, status, timeout_ns));
}
// 16 or 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
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
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait_regs(r);
}
// GELU of two values, y Phi(y) = max(y, 0) - z Q(z) with z = |y| and Q(z) = erfc(z / sqrt 2) / 2, the
// normal distribution's tail.  Q(z) = exp(-z^2 / 2) R(z), and R falls smoothly like 1 / z: in t = 1 / (1 + 0.301 z)
// (the substitution of Hastings' formulas, Abramowitz & Stegun 7.1.26) it is t times a polynomial, of
// degree 7 here, fitted by weighted least squares with Lawson's weights to the least relative error over
// 0 <= z <= 13.5: 1.5e-7 with rounded coefficients.  With the FP32 steps the result is within half a unit
// in its last place + (20 + 1.5 z^2) 2^-24 z Q(z), so it keeps its leading digits in all of the left tail, where formulas for erf
// lose them.  (7.1.28, with one special-function operation a value instead of two, takes 4096 x 3072 x 768
// 18.3 us instead of 20.3, but errs by up to 7e-7, and by 5 % at y = -5.  One reciprocal for both values: 21.0.)
// z is kept at 30, where Q is zero, so that an infinity gives max(y, 0); NaN stays NaN.
__device__ __forceinline__ void gelu2(float& y0, float& y1) {
    const uint64_t z = f2_pack(fminf(fabsf(y0), 30.0f), fminf(fabsf(y1), 30.0f));
    const auto two = [](float v) { return f2_pack(v, v); };
    float a, b, c, d;
    f2_unpack(f2_fma(z, two(0.301f), two(1.0f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(a));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(b));
    const uint64_t t = f2_pack(c, d);
    // -R(z) / t
    uint64_t p = f2_fma(two(-0.036172338f), t, two(0.15756063f));
    p = f2_fma(p, t, two(-0.20416015f));
    p = f2_fma(p, t, two(0.05221945f));
    p = f2_fma(p, t, two(-0.1279228f));
    p = f2_fma(p, t, two(-0.10035842f));
    p = f2_fma(p, t, two(-0.12113759f));
    p = f2_fma(p, t, two(-0.12002871f));
    p = f2_mul(p, t);
    // exp(-z^2 / 2) = 2^(-z^2 log2(e) / 2)
    f2_unpack(f2_mul(f2_mul(z, two(-0.72134752f)), z), a, b);
    p = f2_mul(p, f2_pack(ex2_approx(a), ex2_approx(b)));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(c) : "f"(y0));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(d) : "f"(y1));
    f2_unpack(f2_fma(z, p, f2_pack(c, d)), y0, y1);
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// alpha' acc + bias -> act -> + beta R -> cast of C rows m0 .. m0 + CN - 1 (those below M) at this lane's
// column n: the rows' addresses are the warp's, a lane adds its own offset (32 bits: N stays below 2^30).
template <int CN>
__device__ __forceinline__ void f4_store(const EpiParams& e, float alpha, float bias, int64_t m0, uint32_t n,
                                         float (&v)[CN]) {
    static_assert(CN % 2 == 0, "pairs");
    const int live = static_cast<int>(min(static_cast<int64_t>(CN), e.M - m0));
    if (n >= static_cast<uint32_t>(e.N) || live <= 0) return;
    float r[CN];
    if (e.R) {
        const char* p = reinterpret_cast<const char*>(e.R + m0 * e.ldr);
#pragma unroll
        for (int j = 0; j < CN; ++j) {
            r[j] = j < live ? __ldg(reinterpret_cast<const float*>(p + n * 4u)) : 0.0f;
            p += e.ldr * 4;
        }
    }
    const uint64_t a2 = f2_pack(alpha, alpha), b2 = f2_pack(bias, bias);
#pragma unroll
    for (int j = 0; j < CN; j += 2) f2_unpack(f2_fma(f2_pack(v[j], v[j + 1]), a2, b2), v[j], v[j + 1]);
    if (e.act == GEMM_ACT_GELU_ERF) {
#pragma unroll
        for (int j = 0; j < CN; j += 2) gelu2(v[j], v[j + 1]);
    } else if (e.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < CN; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    }
    if (e.R) {
#pragma unroll
        for (int j = 0; j < CN; ++j) v[j] = fmaf(e.beta, r[j], v[j]);
    }
    const int64_t size = e.out_dtype == GEMM_F32 ? 4 : 2;
    char* c = static_cast<char*>(e.C) + m0 * e.ldc * size;
    const int64_t step = e.ldc * size;
    if (size == 4) {
        if (live == CN) {
#pragma unroll
            for (int j = 0; j < CN; ++j, c += step) *reinterpret_cast<float*>(c + n * 4u) = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < CN; ++j, c += step)
                if (j < live) *reinterpret_cast<float*>(c + n * 4u) = v[j];
        }
    } else {
        uint32_t w[CN / 2];  // two values in 16 bits each
#pragma unroll
        for (int j = 0; j < CN; j += 2) {
            if (e.out_dtype == GEMM_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[j], v[j + 1]);
                w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v[j], v[j + 1]);
                w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        if (live == CN) {
#pragma unroll
            for (int j = 0; j < CN; ++j, c += step)
                *reinterpret_cast<uint16_t*>(c + n * 2u) = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
        } else {
#pragma unroll
            for (int j = 0; j < CN; ++j, c += step)
                if (j < live)
                    *reinterpret_cast<uint16_t*>(c + n * 2u) = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
        }
    }
}

template <int BN, int STAGES, int FMT, int MODE>
constexpr int f4_smem() {
    // ring; full / empty per stage; tfull x2, tempty x2, drain, pair exit x2; copy counts; slot, flag
    return 1024 + STAGES * F4Layout<BN, FMT, MODE>::STAGE_ALIGN + (2 * STAGES + 7) * 8 + 32 + 16;
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

// alpha gA gB, rounded once (a partial product may lie outside FP32).
__device__ __forceinline__ float f4_alpha(const F4Args& a) {
    double f = a.e.alpha;
    if (a.gw) f *= static_cast<double>(__ldg(a.gw));
    if (a.gx) f *= static_cast<double>(__ldg(a.gx));
    return static_cast<float>(f);
}

// F4_SPLIT: one tile per cluster, K divided over its CTAs.  Else persistent, a
// CTA (pair) taking one tile after another.
template <int BN, int STAGES, int FMT, int MODE>
__global__ void __launch_bounds__(F4Layout<BN, FMT, MODE>::THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                    const F4Args args) {
    using L = F4Layout<BN, FMT, MODE>;
    constexpr bool PAIR = L::PAIR, SPLIT = MODE == F4_SPLIT;
    static_assert(STAGES <= 8, "copy counts hold 8 stages");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * L::STAGE_ALIGN);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;  // [2]
    uint64_t* tempty = tfull + 2;      // [2] an accumulator is read (overlapping ones: [0], the shared part)
    uint64_t* drain = tempty + 2;
    uint64_t* oreport = drain + 1;     // pair exit: the odd CTA's copy counts are ready (even CTA's)
    uint64_t* pdone = oreport + 1;     // pair exit: the even CTA saw them all land (odd CTA's)
    uint32_t* uses = reinterpret_cast<uint32_t*>(pdone + 1);  // [8] copies issued per stage
    uint32_t* tmem_slot = uses + 8;
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = MODE == F4_ONE ? 0u : cluster_ctarank();

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&tfull[0]), 1);
        mbar_init(smem_u32(&tfull[1]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&tempty[i]), (PAIR ? 2 : 1) * L::EW);
        mbar_init(smem_u32(drain), 1);
        mbar_init(smem_u32(oreport), 1);
        mbar_init(smem_u32(pdone), 1);
        for (int i = 0; i < 8; ++i) uses[i] = 0u;
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        if (PAIR)
            tmem_alloc_pair(smem_u32(tmem_slot), L::TMEM_COLS);
        else
            tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the peer's barriers are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t tmo = args.timeout_ns;

    uint32_t splits = 1;
    if (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    const int64_t t_end = args.n_tiles * args.m_tiles;
    const int64_t t_begin = SPLIT ? blockIdx.x / splits : PAIR ? blockIdx.x >> 1 : blockIdx.x;
    const int64_t t_step = SPLIT ? t_end : PAIR ? gridDim.x >> 1 : gridDim.x;
    const int kb_lo = SPLIT ? static_cast<int>(static_cast<int64_t>(args.k_blocks) * rank / splits) : 0;
    const int kb_hi = SPLIT ? static_cast<int>(static_cast<int64_t>(args.k_blocks) * (rank + 1) / splits)
                            : args.k_blocks;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ producer
            const bool stall = ((args.flags & GEMM_FLAG_TEST_STALL) && blockIdx.x == 0) ||
                               ((args.flags & GEMM_FLAG_TEST_STALL_PEER) && blockIdx.x == 1);
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            bool ok = true;
            for (int64_t t = t_begin; ok && t < t_end; t += t_step) {
                int64_t mt, nt;
                f4_tile(args, t, mt, nt);
                const int32_t wt = static_cast<int32_t>(nt * (L::TILE_W / FW) + (PAIR ? rank : 0));
                const int32_t x0 = static_cast<int32_t>(mt * BN + (PAIR ? rank * L::X_ROWS : 0));
                const int32_t xt = static_cast<int32_t>(mt * BN / 128);
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&empty[s]), ph ^ 1u, abort_flag, args.status, tmo)) {
                        ok = false;
                        break;
                    }
                    armed &= ~(1u << s);
                    if (!(stall && t == t_begin && kb == kb_lo)) {
                        const uint32_t st = smem_u32(smem + s * L::STAGE_ALIGN);
                        // In a pair, both CTAs' boxes of a stage count on the even CTA's full[s].
                        const uint32_t bar = PAIR ? mapa_shared(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                        if (!PAIR || rank == 0)
                            mbar_arrive_expect_tx(smem_u32(&full[s]), (PAIR ? 2 : 1) * L::STAGE_BYTES);
                        const auto load = [&](uint32_t dst, const CUtensorMap* m, int32_t c0, int32_t c1,
                                              int32_t c2) {
                            if (PAIR)
                                tma_load_3d_pair(dst, m, bar, c0, c1, c2);
                            else
                                tma_load_3d(dst, m, bar, c0, c1, c2);
                        };
                        load(st, &tmW, kb * 128, wt * FW, 0);
                        load(st + F_W_TILE, &tmX, kb * 128, x0, 0);
                        const uint32_t dst = st + F_W_TILE + L::X_TILE;
                        // tiles past the matrix arrive as zeros
                        load(dst, &tmSW, 0, kb * L::CT, wt);
                        load(dst + L::SFW_BYTES, &tmSX, 0, kb * L::CT, xt);
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                        if (PAIR) uses[s] += 1u;
                    }
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (PAIR) {
                // The pair leaves once every copy that either CTA issued has landed
                // (they all count on the even CTA's barriers).  A producer issues
                // use u + 1 of a stage only after use u was consumed, so the
                // copies in flight belong to each stage's last phase: the odd producer
                // reports its counts, and the even one makes that phase complete
                // by accounting for a share that will not come, waits, and answers.
                const uint64_t lim = 3 * tmo + 1000000ull;
                if (rank == 1) {
                    mbar_arrive_cluster(mapa_shared(smem_u32(oreport), 0));
                    if (!mbar_wait_peer(smem_u32(pdone), 0u, lim) && armed) {
                        const uint64_t t0 = globaltimer_ns();  // no answer: a fixed 200 us
                        while (globaltimer_ns() - t0 < 200000ull) {
                        }
                    }
                } else {
                    const bool got = mbar_wait_peer(smem_u32(oreport), 0u, lim);
                    for (int i = 0; i < STAGES; ++i) {
                        if (!got) {
                            if (!ok && (armed & (1u << i)))
                                tc_drain(smem_u32(&full[i]), (armed_par >> i) & 1u, tmo);
                            continue;
                        }
                        const uint32_t ne = uses[i];
                        const uint32_t no = ld_peer_u32(mapa_shared(smem_u32(&uses[i]), 1));
                        const uint32_t n = ne > no ? ne : no;
                        if (n == 0) continue;
                        if (ne == no + 1)
                            mbar_complete_tx(smem_u32(&full[i]), L::STAGE_BYTES);
                        else if (no == ne + 1)
                            mbar_arrive_expect_tx(smem_u32(&full[i]), L::STAGE_BYTES);
                        else if (ne != no)
                            continue;
                        tc_drain(smem_u32(&full[i]), (n - 1) & 1u, tmo);
                    }
                    if (got) mbar_arrive_cluster(mapa_shared(smem_u32(pdone), 1));
                }
            } else if (!ok) {
                for (int i = 0; i < STAGES; ++i)
                    if (armed & (1u << i)) tc_drain(smem_u32(&full[i]), (armed_par >> i) & 1u, tmo);
            }
        }
        __syncwarp();
    } else if (warp == 1 && (!PAIR || rank == 0)) {
        // ---------------------------------------------------- MMA issuer
        // (in a pair, only the even CTA's warp issues).  The whole warp walks the
        // stages, so that addresses and descriptors stay in uniform registers; one
        // elected lane issues.  (With the loop inside a single lane's branch, issuing
        // was the bound: 470 us at 8192^3 nvfp4 against 276 us, before pairs.)
        const bool one = elect_one();
        int s = 0, lt = 0, done = 0;
        uint32_t ph = 0, set = 0;
        bool ok = true, issued = false;
        // descriptors of ring stage 0; a stage is STAGE_ALIGN bytes further on
        const uint32_t ring = smem_u32(smem);
        const uint64_t w_desc = smem_desc_sw128(ring, 16, 1024);
        const uint64_t x_desc = smem_desc_sw128(ring + F_W_TILE, 16, 1024);
        const uint64_t s_desc = sf_desc(ring + F_W_TILE + L::X_TILE);
        const int k_steps = static_cast<int>((args.K + 63) / 64);
        const auto commit = [&](uint64_t* bar) {
            if (PAIR)
                tc_commit_pair(smem_u32(bar), 0x3);
            else
                tc_commit(smem_u32(bar));
        };
        for (int64_t t = t_begin; ok && t < t_end; t += t_step, ++lt) {
            // the accumulator's columns are free: overlapping ones once the tile before has
            // handed back the shared part, else after the tile two before
            const int n_wait = L::OVERLAP ? lt : lt >> 1;  // phases that must be complete
            if (!mbar_wait_warp(smem_u32(&tempty[L::OVERLAP ? 0 : lt & 1]), static_cast<uint32_t>(n_wait ^ 1) & 1u,
                                abort_flag, args.status, tmo)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>((lt & 1) * L::ACC_STEP);
            for (int kb = kb_lo; kb < kb_hi; ++kb) {
                if (!mbar_wait_warp(smem_u32(&full[s]), ph, abort_flag, args.status, tmo)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t off = static_cast<uint64_t>(s * (L::STAGE_ALIGN >> 4));
                const uint32_t sf_t = tmem_base + L::SF_BASE + set * L::SF_COLS;
                set = set + 1 == L::SETS ? 0 : set + 1;
                // The copies below overwrite the scale columns of SETS stages ago: its MMAs must
                // have read them (the stages since keep the tensor cores busy meanwhile).
                static_assert(L::SETS < STAGES, "the stage's barrier has not gone round");
                if (done >= L::SETS) {
                    const int sp = s >= L::SETS ? s - L::SETS : s + STAGES - L::SETS;
                    if (!mbar_wait_warp(smem_u32(&empty[sp]), s >= L::SETS ? ph : ph ^ 1u, abort_flag, args.status,
                                        tmo)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                ++done;
                const int steps = k_steps - kb * 4;  // 4 or more: a whole stage
                if (one) {
                    // TMEM columns of scale tile c: weights at 4c, tokens' row tile x at
                    // 4 (CT + c XT + x).  nvfp4: a tile per step; mxfp4: two steps share
                    // a tile, bytes 0-1 and 2-3
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk > 0 && steps <= kk) break;
                        constexpr int PER = 4 / L::CT;  // steps per scale tile
                        const int c = kk / PER;
                        if (kk % PER == 0) {
                            sf_copy<PAIR>(sf_t + 4 * c, s_desc + off + c * (kFp4TileBytes >> 4));
#pragma unroll
                            for (int x = 0; x < L::XT; ++x)
                                sf_copy<PAIR>(sf_t + 4 * (L::CT + c * L::XT + x),
                                              s_desc + off + ((L::SFW_BYTES * (1 + x) + c * kFp4TileBytes) >> 4));
                        }
                        const uint32_t id = PER == 2 ? (kk & 1) * 2u : 0u;
                        mma_f4<FMT, PAIR>(d, w_desc + off + kk * 2, x_desc + off + kk * 2,
                                          args.idesc | (id << 29) | (id << 4), sf_t + 4 * c,
                                          sf_t + 4 * (L::CT + c * L::XT), (kb > kb_lo || kk > 0) ? 1u : 0u);
                    }
                    commit(&empty[s]);
                }
                issued = true;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if (one) commit(&tfull[lt & 1]);
        }
        if (!ok && issued && one) {
            if (PAIR)
                tc_commit_pair(smem_u32(drain), 0x1);
            else
                tc_commit(smem_u32(drain));
            tc_drain(smem_u32(drain), 0u, tmo);
        }
        __syncwarp();
    } else if (warp >= 2) {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3;
        const int h = (warp - 2) >> 2;         // which of the quarter's warps
        constexpr int CH = BN >= 32 ? 32 : 16;  // columns of a chunk
        constexpr int STEP = CH * (L::EW / 4);  // from one of its chunks to the next
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        const float alpha = f4_alpha(args);
        // K = 0 issued no MMA: the sum is zero
        const bool none = kb_lo == kb_hi;
        int lt = 0;
        for (int64_t t = t_begin; t < t_end; t += t_step, ++lt) {
            int64_t mt, nt;
            f4_tile(args, t, mt, nt);
            const uint32_t n = static_cast<uint32_t>(nt * L::TILE_W + (PAIR ? rank * FW : 0)) + q * 32 + lane;
            const float bias = args.e.bias && n < static_cast<uint32_t>(args.N) ? __ldg(args.e.bias + n) : 0.0f;
            const int buf = lt & 1;
            if (!mbar_wait_warp(smem_u32(&tfull[buf]), static_cast<uint32_t>(lt >> 1) & 1u, abort_flag,
                                args.status, tmo))
                break;
            tc_fence_after();
            // Overlapping accumulators: the shared columns come first (the first one's last
            // 96, the second one's first), within every warp's first chunk, and are handed back as
            // soon as that is read; else the accumulator is, after the last.
            const int start = L::OVERLAP && buf == 0 ? BN - L::OVERLAP : 0;
            static_assert(L::OVERLAP <= STEP, "the shared columns lie in the first chunks");
#pragma unroll 1
            for (int i = CH * h; i < BN; i += STEP) {
                const int c = (start + i) % BN;
                const bool live = SPLIT || mt * BN + c < args.M;
                uint32_t r[CH];
                if (live) tmem_ld_cols(tmem_base + lane_base + static_cast<uint32_t>(buf * L::ACC_STEP + c), r);
                if (!SPLIT && (L::OVERLAP ? i < STEP : i + STEP >= BN)) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        uint64_t* bar = &tempty[L::OVERLAP ? 0 : buf];
                        if (PAIR)
                            mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
                        else
                            mbar_arrive(smem_u32(bar));
                    }
                }
                if (!live) continue;
#pragma unroll
                for (int k = 0; k < CH; k += 16) {
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = none ? 0.0f : __uint_as_float(r[k + j]);
                    if (SPLIT) {
                        // every MMA of this CTA is done: the ring is free for the partial sums,
                        // four columns of a lane together
                        float4* part = reinterpret_cast<float4*>(smem) + ((c + k) / 4) * FW + q * 32 + lane;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[j * FW] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else {
                        f4_store<16>(args.e, alpha, bias, mt * BN + c + k, n, v);
                        __syncwarp();
                    }
                }
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= 2) {
            // (a CTA that gave up leaves its sums undefined; the status says so)
            int64_t mt, nt;
            f4_tile(args, t_begin, mt, nt);
            const int q = warp & 3, h = (warp - 2) >> 2;
            const uint32_t n = static_cast<uint32_t>(nt * FW) + q * 32 + lane;
            const float alpha = f4_alpha(args);
            const float bias = args.e.bias && n < static_cast<uint32_t>(args.N) ? __ldg(args.e.bias + n) : 0.0f;
            const int cols = static_cast<int>(min(static_cast<int64_t>(BN), args.M - mt * BN));
            const uint32_t part = smem_u32(smem) + (q * 32 + lane) * 16;
            // four columns at a time in turn over the cluster's warps of this quarter
            const int step = 4 * static_cast<int>(splits) * (L::EW / 4);
            for (int c = 4 * (static_cast<int>(rank) * (L::EW / 4) + h); c < cols; c += step) {
                float4 p[8];
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    p[k] = k < splits ? ld_cluster_f4(mapa_shared(part + (c / 4) * FW * 16, k))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float v[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                    v[0] += p[k].x;
                    v[1] += p[k].y;
                    v[2] += p[k].z;
                    v[3] += p[k].w;
                }
                f4_store<4>(args.e, alpha, bias, mt * BN + c, n, v);
            }
        }
        __syncwarp();
    }
    __syncwarp();
    if (MODE != F4_ONE) cluster_sync();  // no CTA leaves while another reads or signals it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (PAIR)
            tmem_dealloc_pair(tmem_base, L::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
}

struct F4Maps {
    CUtensorMap w, x, sw, sx;
};

template <int BN, int STAGES, int FMT, int MODE>
cudaError_t launch_f4(const F4Maps& m, const F4Args& a, int splits, int num_sms, cudaStream_t st) {
    using L = F4Layout<BN, FMT, MODE>;
    auto k = fp4_gemm_kernel<BN, STAGES, FMT, MODE>;
    constexpr int smem = f4_smem<BN, STAGES, FMT, MODE>();
    static_assert(smem <= kMaxDynSmem, "shared memory");
    static_assert(MODE != F4_SPLIT || STAGES * L::STAGE_ALIGN >= BN * FW * 4, "partial sums fit the ring");
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
    const int64_t grid = MODE == F4_SPLIT  ? tiles * splits
                         : MODE == F4_PAIR ? 2 * std::min<int64_t>(tiles, num_sms / 2)
                                           : std::min<int64_t>(tiles, num_sms);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (MODE != F4_ONE) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(MODE == F4_PAIR ? 2 : splits);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, m.w, m.x, m.sw, m.sx, a);
}

template <int BN, int STAGES, int MODE>
cudaError_t launch_fmt(int fmt, const F4Maps& m, const F4Args& a, int splits, int num_sms, cudaStream_t st) {
    return fmt == GEMM_MXFP4 ? launch_f4<BN, STAGES, GEMM_MXFP4, MODE>(m, a, splits, num_sms, st)
                             : launch_f4<BN, STAGES, GEMM_NVFP4, MODE>(m, a, splits, num_sms, st);
}
template <int BN, int STAGES>
cudaError_t launch_bn(int fmt, const F4Maps& m, const F4Args& a, int splits, int num_sms, cudaStream_t st) {
    return splits > 1 ? launch_fmt<BN, STAGES, F4_SPLIT>(fmt, m, a, splits, num_sms, st)
                      : launch_fmt<BN, STAGES, F4_ONE>(fmt, m, a, 1, num_sms, st);
}

}  // namespace

int launch_fp4_gemm(const Fp4Config& c, int fmt, const Fp4Operand& A, const Fp4Operand& B, int64_t K,
                    const EpiParams& e, const LaunchCtx& lc) {
    const bool pair = c.bn == 256;
    const int tile_w = pair ? 2 * FW : FW;
    F4Args a{};
    a.M = e.M;
    a.N = e.N;
    a.K = K;
    a.gw = B.tensor_scale;
    a.gx = A.tensor_scale;
    a.n_tiles = (e.N + tile_w - 1) / tile_w;
    a.m_tiles = (e.M + c.bn - 1) / c.bn;
    a.k_blocks = static_cast<int>((K + F_KB - 1) / F_KB);
    a.raster = 8;
    a.e = e;
    a.status = lc.status;
    a.timeout_ns = lc.timeout_ns;
    a.flags = lc.flags;
    // instruction descriptor: E2M1 operands (1), scale type (1: UE8M0), N, M
    a.idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(c.bn >> 3) << 17) |
              ((fmt == GEMM_MXFP4 ? 1u : 0u) << 23) | (static_cast<uint32_t>(tile_w >> 7) << 27);
    F4Maps m{};
    if (K > 0) {
        const int64_t rb = fp4_row_bytes(K);
        const int64_t ct = fp4_col_tiles(fmt, K);
        const uint32_t box_ct = static_cast<uint32_t>(F_KB / (4 * fp4_block(fmt)));
        int rc = tmap_encode_rows_u8(&m.w, B.codes, rb, e.N, FW);
        if (rc == GEMM_OK)
            rc = tmap_encode_rows_u8(&m.x, A.codes, rb, e.M, static_cast<uint32_t>(pair ? c.bn / 2 : c.bn));
        if (rc == GEMM_OK)
            rc = tmap_encode_tiles(&m.sw, B.scales, ct, fp4_row_tiles(e.N), kFp4TileBytes, box_ct, 1);
        if (rc == GEMM_OK)
            rc = tmap_encode_tiles(&m.sx, A.scales, ct, fp4_row_tiles(e.M), kFp4TileBytes, box_ct,
                                   static_cast<uint32_t>((c.bn + 127) / 128));
        if (rc != GEMM_OK) return rc;
    }
    cudaError_t ce;
    switch (c.bn) {
        case 16: ce = launch_bn<16, 8>(fmt, m, a, c.splits, lc.num_sms, lc.stream); break;
        case 32: ce = launch_bn<32, 8>(fmt, m, a, c.splits, lc.num_sms, lc.stream); break;
        case 64: ce = launch_bn<64, 7>(fmt, m, a, c.splits, lc.num_sms, lc.stream); break;
        case 128: ce = launch_bn<128, 6>(fmt, m, a, c.splits, lc.num_sms, lc.stream); break;
        case 256:  // as many stages as shared memory holds (mxfp4's 35 KB: 6, 184 us at 8192^3 instead of 187)
            ce = fmt == GEMM_MXFP4 ? launch_f4<256, 6, GEMM_MXFP4, F4_PAIR>(m, a, 1, lc.num_sms, lc.stream)
                                   : launch_f4<256, 5, GEMM_NVFP4, F4_PAIR>(m, a, 1, lc.num_sms, lc.stream);
            break;
        default: return GEMM_ERR_UNSUPPORTED;
    }
    return cuda_status(ce);
}

// Clusters of `splits` CTAs (one CTA per SM) that run at a time: a cluster stays within a
// part of the GPU, so the larger ones leave SMs over (152 SMs hold 76, 36 and 15 of 2, 4 and 8).
int64_t clusters_at_once(int splits, int num_sms) {
    return splits == 1 ? num_sms : splits == 2 ? num_sms / 2 : splits == 4 ? num_sms / 4 - num_sms / 76 : num_sms / 10;
}

// Up to 64 tokens: the narrowest of 16, 32, 64 that holds them all (a stage streams the same
// weights with any of them), K split over a cluster of 2, 4 or 8 while all tiles run at once.
// Above: the cheapest of 128 x 128 tiles, those with K split, and CTA pairs on 256 x 256, by a
// model in ns: a stage of 256 K elements takes 300 on 128 x 128 (the bytes from L2 bound it: 36 KB
// per SM) and 360 on a pair for four times the area (38 KB per SM); a tile's stages hide the one
// before's epilogue, or wait for it (1500, 3000); launch, fill and last epilogue as measured.
Fp4Config fp4_choose(int64_t M, int64_t N, int64_t K, int num_sms) {
    Fp4Config best{};
    best.bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    best.splits = 1;
    const int64_t n_tiles = (N + FW - 1) / FW, kbs = (K + F_KB - 1) / F_KB;
    const int64_t tiles = n_tiles * ((M + best.bn - 1) / best.bn);
    if (tiles == 0) return best;
    const auto waves = [](int64_t t, int64_t at_once) { return (t + at_once - 1) / at_once; };
    int64_t cost = waves(tiles, num_sms) * std::max<int64_t>(300 * kbs, 1500) + 2500;
    for (int s = 2; s <= 8 && s <= kbs; s *= 2) {
        if (tiles > clusters_at_once(s, num_sms)) break;
        const int64_t c = 300 * ((kbs + s - 1) / s) + 3500;
        if (c < cost || M <= 64) {
            cost = c;
            best.splits = s;
        }
    }
    if (M > 64) {
        const int64_t pairs = ((N + 255) / 256) * ((M + 255) / 256);
        const int64_t c = waves(pairs, num_sms / 2) * std::max<int64_t>(360 * kbs, 3000) + 3500;
        if (num_sms >= 2 && c < cost) return Fp4Config{256, 1};
    }
    return best;
}

}  // namespace g13
