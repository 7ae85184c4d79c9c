// w4_tc.cu -- products of 17 to 64 tokens with 4-bit weights on the tensor cores (tcgen05).
//
// The weights' rows are the 128 rows of a tile and the tokens its columns.  A step is 128 columns of K.  Eight warps turn its
// codes into q - z, whole numbers of at most four bits and a sign and so exact in X's own type, and write them to shared memory
// as the 128-byte-swizzled rows that tcgen05.mma reads; the tokens' values come beside them as they are (cp.async).  No
// activation and no weight is rounded.  The scales stay out of the product: each group's sum (of a step at most) has
// TMEM columns of its own, others read them, a thread to a row, and add scale * sum in FP32.
//
//   4 warps       sums: TMEM to registers, times the row's scale
//   8 or 16 warps codes and tokens to shared memory, in a ring, eight to a step: full[s] counts their arrivals.  Up to 32
//                 tokens two sets of eight take steps in turn; with more the sums' registers leave room for one
//   the last      one lane issues the MMAs; commits free ring stages (empty[s]) and hand sums over (tfull[b])
//
// Measured at 16384 x 8192, BF16, groups of 128 / 64 / 32: 17 tokens 33.6 / 40.1 / 68.1 us; 64 tokens 45.5 (128) and 68.2
// (32); the bytes would take 10.8.  A step is 2660 warp instructions at 17 tokens and 3130 at 64, which take 77 % and 69 % of the
// issue slots of the 128 SMs that have a tile (24 have none), and the tensor pipes 15 % and 22 %: the instructions bound the
// first, and them together with the way of a step through a ring of three stages the second.  One set of
// producers: 45 us at 32 tokens; weights in TMEM, tokens by copies of four bytes: 84 at 64.
//
// A CTA has one tile, or a cluster of two to eight shares its K and adds the CTAs' sums in rank order through
// distributed shared memory.  Every wait is bounded; after a timeout the tile's results are NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "ptx.cuh"
#include "w4.cuh"

namespace g13 {
namespace {

constexpr int TC_WRITERS = 8;          // producer warps of a step, 16 rows each
constexpr int TC_AHEAD = 4;            // steps whose codes are in registers, and tokens asked for
constexpr int TC_SCALES = 4;           // steps of scales in registers
constexpr int TC_A_BYTES = 128 * 256;  // 128 rows x 128 columns, two halves of 64 columns
constexpr int TC_SUM_ROW = 128 + 4;
constexpr uint64_t TC_DRAIN_NS = 2000000000ull;  // what was issued is waited for this long at most

struct W4TcPlan {
    int steps, blocks, tiles, groups;  // tiles: blocks of 16 rows
    uint32_t inv;                      // reciprocal of group / 32
    uint32_t idesc;
    uint64_t timeout_ns;               // of each wait
    uint32_t flags;
};

template <int TOK, int NG>
struct TcLayout {
    static constexpr int TURNS = TOK == 64 ? 1 : 2;           // sets of producers, which take steps in turn
    static constexpr int AHEAD = TC_AHEAD / TURNS;            // of a producer's own steps
    static constexpr int STAGES = TOK == 64 ? 3 : 4;          // of codes
    static constexpr int X_STAGES = STAGES + TC_AHEAD;        // of tokens: these are asked for that much earlier
    static constexpr int X_BYTES = TOK * 256;
    static constexpr int RING = STAGES * TC_A_BYTES + X_STAGES * X_BYTES;
    static constexpr int EW = 4;                              // warps with sums
    static constexpr int THREADS = 32 * (EW + TC_WRITERS * TURNS + 1);
    static constexpr int BUFS = 4 * NG * TOK <= 512 ? 4 : 2;  // of steps' sums, TOK TMEM columns a group
    static constexpr int COLS = BUFS * NG * TOK;
    static constexpr int SMEM = 1024 + RING + (2 * STAGES + 2 * BUFS + 1) * 8 + 16;
    static_assert(TOK % 32 == 0 && COLS <= 512 && SMEM <= kW4Smem, "TMEM, shared memory");
    static_assert(TOK * TC_SUM_ROW * 4 <= RING, "the sums lie where the ring was");
};

// Eight codes less their zero, columns in order, as 16-bit numbers.  FP16: 1024 + q less 1024 + z; in the second lowest
// place 1024 + 16 q, of which a 16th less 64 + z.  BF16 holds 128 + q only, so that place is shifted down first.
template <bool BF16>
struct Zero {
    uint32_t low, high;
    __device__ __forceinline__ explicit Zero(uint32_t z) {
        const uint32_t two = z | z << 16;
        low = two | (BF16 ? 0x43004300u : 0x64006400u);
        high = two << 4 | 0xD400D400u;  // -(64 + z)
    }
};
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b, __half2) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b, __nv_bfloat162) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sixteenth(uint32_t a, uint32_t b) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(0.0625f), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool BF16>
__device__ __forceinline__ uint4 numbers(uint32_t w, const Zero<BF16>& z) {
    constexpr uint32_t LOW = 0x000F000Fu, HIGH = 0x00F000F0u;
    if (BF16) {
        constexpr uint32_t M = 0x43004300u;
        const __nv_bfloat162 t{};
        return make_uint4(less((w & LOW) | M, z.low, t), less((w >> 4 & LOW) | M, z.low, t),
                          less((w >> 8 & LOW) | M, z.low, t), less((w >> 12 & LOW) | M, z.low, t));
    }
    constexpr uint32_t M = 0x64006400u;
    const __half2 t{};
    const uint32_t u = w >> 8;
    return make_uint4(less((w & LOW) | M, z.low, t), sixteenth((w & HIGH) | M, z.high), less((u & LOW) | M, z.low, t),
                      sixteenth((u & HIGH) | M, z.high));
}

template <int TOK, int NG, bool BF16>
__global__ void __launch_bounds__(TcLayout<TOK, NG>::THREADS, 1) w4_tc_kernel(const __grid_constant__ W4Args a, const __grid_constant__ W4TcPlan plan) {
    using L = TcLayout<TOK, NG>;
    constexpr int TURNS = L::TURNS, AHEAD = L::AHEAD, STAGES = L::STAGES, EW = L::EW, MMA_WARP = EW + TC_WRITERS * TURNS;
    extern __shared__ uint8_t tc_raw[];
    uint8_t* smem = tc_raw + ((1024 - (smem_u32(tc_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::RING);
    uint8_t* tokens = smem + STAGES * TC_A_BYTES;
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + L::BUFS;
    uint64_t* drain = tempty + L::BUFS;
    uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ranks, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), TC_WRITERS);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < L::BUFS; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), EW);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) tmem_alloc(smem_u32(slot), L::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    const int tile = static_cast<int>(blockIdx.x / ranks);
    const int first = static_cast<int>(static_cast<uint32_t>(plan.steps) * rank / ranks);
    const int steps = static_cast<int>(static_cast<uint32_t>(plan.steps) * (rank + 1) / ranks) - first;
    // A whole warp's wait: the same answer in every lane, so that none goes on alone.
    const auto wait = [&](uint64_t& bar, uint32_t parity) {
        return mbar_wait_warp(smem_u32(&bar), parity, abort_flag, nullptr, plan.timeout_ns);
    };
    // the group of piece h (of NG) of step j
    const auto group = [&](int j, int h) {
        return min(over(static_cast<uint32_t>((first + j) * 4 + h * (4 / NG)), plan.inv), plan.groups - 1);
    };
    float sums[TOK];  // (of the first warps)

    if (warp >= EW && warp < MMA_WARP) {
        // ---- codes and tokens: a warp has 16 of the tile's rows
        const int pw = (warp - EW) % TC_WRITERS, turn = (warp - EW) / TC_WRITERS, tid = pw * 32 + lane, rb = tile * 8 + pw, r = lane >> 2, c = lane & 3;
        const bool live = rb < plan.tiles;
        const uint8_t* codes = a.codes + (static_cast<int64_t>(rb) * plan.blocks + first * 2) * 512 + lane * 16;
        const uint16_t* zeros = a.zeros ? reinterpret_cast<const uint16_t*>(a.zeros) + static_cast<int64_t>(rb) * plan.groups * 8 + r
                                        : &kEights;
        const int zero_step = a.zeros ? 8 : 0;
        const uint16_t* x = static_cast<const uint16_t*>(a.x);
        struct Ahead {
            uint4 lo, hi;
            uint32_t z[NG];
        } ring[AHEAD] = {};
        const auto load = [&](Ahead& b, int j) {
            const bool on = live && j < steps;
            const uint8_t* p = codes + static_cast<int64_t>(j) * 1024;
            ld_codes(b.lo, p, on);
            // (past the row's end any codes will do: the tokens' values there are zeros)
            ld_codes(b.hi, p + 512, on && (first + j) * 2 + 1 < plan.blocks);
#pragma unroll
            for (int h = 0; h < NG; ++h) ld_nc16(b.z[h], zeros + static_cast<int64_t>(group(j, h)) * zero_step, on);
        };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) load(ring[d], turn + d * TURNS);
        // of stage s: what this lane's words are in row r, and 8 rows on
        const uint32_t row = static_cast<uint32_t>(pw * 16 + r) * 128;
        // (lanes of odd rows write the other half first, so that eight lanes meet all banks)
        const bool odd = r & 1;
        const uint32_t at0 = row + ((c + (odd ? 4 : 0)) ^ r) * 16, at1 = row + ((c + (odd ? 0 : 4)) ^ r) * 16;
        const auto arrive = [&](int s) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&full[s]));
        };
        // the tokens of step j, into stage xs of theirs; a group of copies in any case
        const auto fetch = [&](int j, int xs) {
            uint8_t* stage = tokens + xs * L::X_BYTES;
            const int64_t k = static_cast<int64_t>(first + j) * 128 + (tid & 15) * 8, left = a.K - k;
            const int ch = tid & 15;
            if (j < steps) {
#pragma unroll
                for (int i = 0; i < TOK / 16; ++i) {
                    const int t = (tid >> 4) + i * 16;
                    const bool on = t < a.M && left > 0;
                    cp_async_16z(smem_u32(stage + (ch >> 3) * (TOK * 128) + t * 128 + (((ch & 7) ^ (t & 7)) * 16)),
                                 on ? x + t * a.ldx + k : x, on ? static_cast<uint32_t>(min(left, static_cast<int64_t>(8))) * 2u : 0u);
                }
            }
            cp_async_commit();
        };
        int xs = turn;  // the next stage of tokens to fill
        const auto next_xs = [&] { xs = xs + TURNS >= L::X_STAGES ? xs + TURNS - L::X_STAGES : xs + TURNS; };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            fetch(turn + d * TURNS, xs);
            next_xs();
        }
        bool ok = true;
        int s = turn;
        uint32_t parity = 1;
        for (int j0 = turn; j0 < steps; j0 += TC_AHEAD) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int j = j0 + d * TURNS;
                if (j >= steps) continue;
                // Lanes wait one by one (a vote on the answers costs up to 4 %, 64 x 16384 x 8192).  One whose wait ran out
                // does no more, but meets the others, which may be in arrive, once a step to the end.
                if (ok) ok = mbar_wait_bounded(smem_u32(&empty[s]), parity, abort_flag, nullptr, plan.timeout_ns);
                if (!ok) {
                    __syncwarp();
                    continue;
                }
                uint8_t* stage = smem + s * TC_A_BYTES;
                const Ahead& b = ring[d];
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // 64 columns each; word pairs: 32 columns, rows r and r + 8
                    const uint4 v = h ? b.hi : b.lo;
                    const uint32_t z0 = b.z[h * NG / 2], z1 = b.z[NG == 4 ? h * 2 + 1 : h * NG / 2];
                    const uint32_t za = odd ? z1 : z0, zb = odd ? z0 : z1;
                    uint8_t* to = stage + h * (TC_A_BYTES / 2);
                    *reinterpret_cast<uint4*>(to + at0) = numbers<BF16>(odd ? v.z : v.x, Zero<BF16>(za & 0xFFu));
                    *reinterpret_cast<uint4*>(to + at0 + 1024) = numbers<BF16>(odd ? v.w : v.y, Zero<BF16>(za >> 8 & 0xFFu));
                    *reinterpret_cast<uint4*>(to + at1) = numbers<BF16>(odd ? v.x : v.z, Zero<BF16>(zb & 0xFFu));
                    *reinterpret_cast<uint4*>(to + at1 + 1024) = numbers<BF16>(odd ? v.y : v.w, Zero<BF16>(zb >> 8 & 0xFFu));
                }
                load(ring[d], j + TC_AHEAD);
                cp_async_wait_group<AHEAD - 1>();  // this step's tokens
                arrive(s);
                // (the stage of empty[s] was read by the products of step j - STAGES, and so were these tokens')
                fetch(j + TC_AHEAD, xs);
                next_xs();
                s += TURNS;
                if (s >= STAGES) s -= STAGES, parity ^= 1;
            }
        }
        cp_async_wait_all();
    } else if (warp == MMA_WARP) {
        // The whole warp walks the steps, so that addresses and descriptors stay in uniform registers, and one lane issues
        // (all of it in one lane's branch: 140 cycles to an MMA, 44 us at 16 x 16384 x 8192).
        const bool one = elect_one();
        const uint64_t ad0 = smem_desc_sw128(smem_u32(smem), 16, 1024), bd0 = smem_desc_sw128(smem_u32(tokens), 16, 1024);
        bool ok = true;
        int s = 0, xs = 0;
        uint32_t parity = 0;
        const int issued = (plan.flags & GEMM_FLAG_TEST_STALL) && blockIdx.x == 0 ? 0 : steps;
        for (int j = 0; j < issued && ok; ++j) {
            const int b = j % L::BUFS;
            ok = wait(tempty[b], (j / L::BUFS & 1) ^ 1) && wait(full[s], parity);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = ad0 + static_cast<uint64_t>(s * (TC_A_BYTES >> 4)), bd = bd0 + static_cast<uint64_t>(xs * (L::X_BYTES >> 4));
            if (one) {
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 columns each
                    tc_mma_f16(tmem + (b * NG + k * NG / 8) * TOK, ad + (((k >> 2) * (TC_A_BYTES / 2) + (k & 3) * 32) >> 4),
                               bd + (((k >> 2) * (TOK * 128) + (k & 3) * 32) >> 4), plan.idesc, k % (8 / NG) != 0);
                tc_commit(smem_u32(&empty[s]));
                tc_commit(smem_u32(&tfull[b]));
            }
            if (++s == STAGES) s = 0, parity ^= 1;
            if (++xs == L::X_STAGES) xs = 0;
        }
        if (one) {
            tc_commit(smem_u32(drain));
            // (what was issued ends by itself; a bounded wait without the abort flag)
            volatile uint32_t none = 0;
            mbar_wait_bounded(smem_u32(drain), 0, &none, nullptr, TC_DRAIN_NS);
        }
        __syncwarp();
    } else {
        // ---- sums of row warp * 32 + lane
        const int row = warp * 32 + lane, rb = tile * 8 + row / 16;
        const bool live = rb < plan.tiles;
        const uint16_t* scales = static_cast<const uint16_t*>(a.scales) + static_cast<int64_t>(rb) * plan.groups * 16 + row % 8 * 2 + row % 16 / 8;
        uint32_t ring[TC_SCALES][NG] = {};
        const auto load = [&](uint32_t(&v)[NG], int j) {
#pragma unroll
            for (int h = 0; h < NG; ++h) ld_nc16(v[h], scales + group(j, h) * 16, live && j < steps);
        };
#pragma unroll
        for (int i = 0; i < TOK; ++i) sums[i] = 0.0f;
#pragma unroll
        for (int d = 0; d < TC_SCALES; ++d) load(ring[d], d);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        bool ok = true;
        for (int j0 = 0; ok && j0 < steps; j0 += TC_SCALES) {
#pragma unroll
            for (int d = 0; d < TC_SCALES; ++d) {
                const int j = j0 + d;
                if (!ok || j >= steps) continue;
                const int b = d % L::BUFS;
                ok = wait(tfull[b], j / L::BUFS & 1);
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < NG; ++h) {
                    const float s = BF16 ? __uint_as_float(ring[d][h] << 16)
                                         : __half2float(__ushort_as_half(static_cast<unsigned short>(ring[d][h])));
#pragma unroll
                    for (int n = 0; n < TOK; n += 32) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(lanes + (b * NG + h) * TOK + n, v);
                        tmem_ld_wait_regs(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sums[n + i] = fmaf(s, __uint_as_float(v[i]), sums[n + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[b]));
                load(ring[d], j + TC_SCALES);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    // ---- the sums to shared memory, where the ring was, and the CTAs' shares of them added in rank order
    float* all = reinterpret_cast<float*>(smem);  // [token][row]
    const int tok = static_cast<int>(a.M);
    if (warp < EW) {
        const bool failed = *abort_flag != 0;
#pragma unroll
        for (int t = 0; t < TOK; ++t)
            if (t < tok) all[t * TC_SUM_ROW + warp * 32 + lane] = failed ? __int_as_float(0x7FFFFFFF) : sums[t];
    }
    if (ranks > 1)
        cluster_sync();
    else
        __syncthreads();
    for (int i = static_cast<int>(rank) * L::THREADS + threadIdx.x; i < tok * 32; i += L::THREADS * static_cast<int>(ranks)) {
        const int t = i >> 5, row = (i & 31) * 4;
        const float* p = all + t * TC_SUM_ROW + row;
        float4 v = *reinterpret_cast<const float4*>(p);
        if (ranks > 1) {
            v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (uint32_t k = 0; k < ranks; ++k) {
                const float4 o = ld_cluster_f4(mapa_shared(smem_u32(p), k));
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
        }
        w4_store4(a.e, t, static_cast<int64_t>(tile) * 128 + row, v);
    }
    if (ranks > 1) cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == MMA_WARP) tmem_dealloc(tmem, L::COLS);
}

template <int TOK, int NG, bool BF16>
cudaError_t launch(const W4Args& a, int splits, cudaStream_t st) {
    using L = TcLayout<TOK, NG>;
    auto k = w4_tc_kernel<TOK, NG, BF16>;
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    W4TcPlan p{};
    p.steps = static_cast<int>((a.K + 127) / 128);
    p.blocks = static_cast<int>(w4_blocks(a.K));
    p.tiles = static_cast<int>(w4_tiles(a.N));
    p.groups = static_cast<int>(w4_groups(a.K, a.group));
    p.inv = reciprocal(a.group / 32);
    p.timeout_ns = a.timeout_ns;
    p.flags = a.flags;
    // kind::f16: FP32 sums, both operands of X's type and K-major, TOK columns, 128 rows
    const uint32_t type = BF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(TOK >> 3) << 17) | (8u << 24);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + 127) / 128 * splits));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (splits > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(splits);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, a, p);
}

template <int TOK, int NG>
cudaError_t launch_type(const W4Args& a, int splits, cudaStream_t st) {
    return a.dtype == GEMM_BF16 ? launch<TOK, NG, true>(a, splits, st) : launch<TOK, NG, false>(a, splits, st);
}
template <int NG>
cudaError_t launch_tokens(const W4Args& a, int splits, cudaStream_t st) {
    return a.M <= 32 ? launch_type<32, NG>(a, splits, st) : launch_type<64, NG>(a, splits, st);
}

}  // namespace

// From 17 tokens on.  At 17, w4.cu takes 43.4 / 50.1 / 75.8 us instead of the 33.6 / 40.1 / 68.1 above; at 16 it takes
// 31.5 / 35.7 / 44.0 where these kernels take 33.3 / 39.5 / 67.3.  (With few rows and a long K they win earlier:
// 4096 x 14336, 16 tokens, groups of 128, 18.8 us against 22.9.)  Rows of X off 16 bytes go to w4.cu with any number of tokens.
//
// K is divided as a rough model in ns has it: a step 250, a tile's set-up and store 2500, a cluster's barriers and join 1500 more.
int w4_tc_splits(const W4Args& a, int num_sms) {
    if (a.M <= 16 || reinterpret_cast<uintptr_t>(a.x) % 16 != 0 || (a.M > 1 && a.ldx % 8 != 0)) return 0;
    const int64_t steps = (a.K + 127) / 128, tiles = (a.N + 127) / 128;
    if (tiles * 8 > (int64_t(1) << 31) - 1) return 0;
    int best = 1;
    int64_t least = 0;
    for (int s = 1; s <= 8 && s <= steps; s *= 2) {
        const int64_t at_once = std::max<int64_t>(1, clusters_at_once(s, num_sms));
        const int64_t t = (tiles + at_once - 1) / at_once * ((steps + s - 1) / s * 250 + 2500 + (s > 1 ? 1500 : 0));
        if (s == 1 || t < least) least = t, best = s;
    }
    return best;
}

cudaError_t launch_w4_tc(const W4Args& a, int splits, cudaStream_t st) {
    switch (w4_per_step(a.group)) {
        case 1: return launch_tokens<1>(a, splits, st);
        case 2: return launch_tokens<2>(a, splits, st);
        default: return launch_tokens<4>(a, splits, st);
    }
}

}  // namespace g13
