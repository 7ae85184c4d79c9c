// moe.cu -- a mixture-of-experts layer for a few tokens (1 to 64):
//
//   z = x Wr^T;  p = softmax(z) over all experts;  the top_k largest z (ties: the
//   lowest index) with weights p, or p divided by their sum;
//   y = sum_j weight_j  W2[e_j] act(W1[e_j] x)
//   act: GELU or ReLU of I rows, or SwiGLU: silu(gate) * up, gate = rows 0..I-1 of
//   W1[e], up = rows I..2I-1
//
// A few tokens leave two products per weight byte and token: reading the chosen
// experts' weights once is the cost, so everything is laid out to keep those
// loads in flight.  Two kernels:
//
//   router   z in FP32 (one warp per expert and four tokens); copies x into rows
//            padded to 64 elements; clears the counters of the second kernel
//   experts  one CTA of 16 warps per SM, cooperative.  Every CTA works out the
//            routing for itself from z (softmax, top-k by warp-wide maximum
//            reductions, a 64-bit mask of tokens per expert), which is cheaper than
//            another trip through memory.  Then the two products, with one grid
//            barrier between them:
//     up     work units of 16 weight rows of a chosen expert (SwiGLU: 8 gate rows
//            and their 8 up rows, so one thread holds both factors) x 64-element
//            steps along H.  A CTA takes an equal share of the units and its warps
//            equal shares of the units' steps; a unit cut between warps is joined
//            through shared memory, in warp order.
//     down   units (16 output columns, chosen expert), column block major, cut
//            the same way; each warp adds weight * product to its own tile of the
//            output in shared memory.  A block cut between CTAs leaves partial sums
//            in the workspace, and the CTA that arrives last adds them in
//            CTA order: the result does not depend on timing.
//
// Products: mma.sync m16n8k16, weights as the 16 rows and a group of 8 tokens as
// the columns.  The order of k within a step is free as long as both operands share
// it, so a thread takes 32 consecutive bytes of a row (16 values: four MMAs' worth)
// straight from global memory as its fragments; no shared memory, no barrier.
// (tcgen05 would need the weights staged through shared memory, to do arithmetic
// that is far from the bound.)  FP32 accumulation; h = act(...) is rounded to
// the operands' 16-bit type, which the second product needs as its operand.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "epilogue.cuh"
#include "moe.h"
#include "ptx.cuh"

namespace g13 {
namespace {

constexpr int MT = kMoeWarps * 32;   // threads per CTA
constexpr int RT = 256;              // threads per router CTA
constexpr int kMaxDevices = 64;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// How the rows of a weight lie: all on 32 bytes with lengths a multiple of 16 elements, all
// on 16 bytes with multiples of 8, or anyhow.
enum Rows { ROWS_32 = 0, ROWS_16 = 1, ROWS_ANY = 2 };

// Eight consecutive 16-bit values at p, of which the first n (0 to 8) exist; the rest
// are zero.  VEC: p is 16-byte aligned and n is 0 or 8.  Else two aligned 16-byte loads
// of the granules that hold the values (each holds at least one of them), shifted.
template <bool VEC>
__device__ __forceinline__ uint4 ld_row8(const uint16_t* p, int n) {
    if (VEC) return n > 0 ? ld_stream(p) : make_uint4(0, 0, 0, 0);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (n > 0) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const unsigned o = static_cast<unsigned>(at & 15);
        const char* base = reinterpret_cast<const char*>(at - o);
        a = ld_stream(base);
        if (o + 2 * min(n, 8) > 16) b = ld_stream(base + 16);
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (o & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (o & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = __funnelshift_r(w[i], w[i + 1], (o & 2) * 8);
            if (2 * i + 1 >= n) v = 2 * i >= n ? 0u : v & 0xFFFFu;
            w[i] = v;
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return a;
}
// Sixteen of them.
struct Row16 {
    uint32_t v[8];
};
template <int ROWS>
__device__ __forceinline__ Row16 ld_row16(const uint16_t* p, int n) {
    Row16 r;
    if (ROWS == ROWS_32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = 0u;
        if (n > 0)
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3]), "=r"(r.v[4]), "=r"(r.v[5]),
                           "=r"(r.v[6]), "=r"(r.v[7])
                         : "l"(p));
    } else {
        const uint4 a = ld_row8<ROWS == ROWS_16>(p, n), b = ld_row8<ROWS == ROWS_16>(p + 8, n - 8);
        r = Row16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return r;
}

// Equal shares of `total` for `parts` takers, the first ones one longer.
struct Share {
    int q, r;
    __device__ __forceinline__ Share(int total, int parts) : q(total / parts), r(total % parts) {}
    __device__ __forceinline__ int lo(int i) const { return i * q + min(i, r); }
    // The taker of item u (shares that are not empty).
    __device__ __forceinline__ int owner(int u) const {
        const int longer = r * (q + 1);
        return u < longer ? u / (q + 1) : r + (u - longer) / max(q, 1);
    }
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
template <typename T>
__device__ __forceinline__ T cast16(float v);
template <>
__device__ __forceinline__ __half cast16(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 cast16(float v) { return __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                 uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// GELU in its erf form, or ReLU; NaN stays NaN.
__device__ __forceinline__ float moe_act(int act, float y) {
    if (act == GEMM_MOE_GELU) return epi_act(GEMM_ACT_GELU_ERF, y);
    return y < 0.0f ? 0.0f : y;
}

// ------------------------------------------------------------------ router
template <typename T, bool VEC>
__global__ void __launch_bounds__(RT) moe_router_kernel(const MoeArgs a) {
    const gemm_moe_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (every count here stays below 2^31; 64-bit divisions would cost microseconds)
    const int tid = static_cast<int>(blockIdx.x) * RT + threadIdx.x;
    const int nthreads = static_cast<int>(gridDim.x) * RT;
    // counters, padded x, and the padding of h (never written by the up product)
    unsigned* ctr = reinterpret_cast<unsigned*>(a.ws + a.w.bar);
    const int n_ctr = static_cast<int>((a.w.logits - a.w.bar) / 4);
    for (int i = tid; i < n_ctr; i += nthreads) ctr[i] = 0u;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    uint16_t* xp = reinterpret_cast<uint16_t*>(a.ws + a.w.x);
    const int hp = static_cast<int>(a.w.hp), H = static_cast<int>(d.H);
    for (int i = tid; i < static_cast<int>(d.T) * hp; i += nthreads) {
        const int t = i / hp, k = i - t * hp;
        xp[i] = k < H ? x[t * d.ldx + k] : uint16_t(0);
    }
    uint16_t* h = reinterpret_cast<uint16_t*>(a.ws + a.w.h);
    const int pad = static_cast<int>(a.w.ip - d.I);
    for (int i = tid; i < static_cast<int>(d.T * d.top_k) * pad; i += nthreads)
        h[static_cast<int64_t>(i / pad) * a.w.ip + d.I + i % pad] = 0;

    // z: a warp takes one expert and four tokens
    const int unit = static_cast<int>(blockIdx.x) * (RT / 32) + warp;
    const int t0 = unit / static_cast<int>(d.E) * 4;
    const int64_t e = unit % static_cast<int>(d.E);
    if (t0 >= d.T) return;
    const int nt = min(4, static_cast<int>(d.T) - t0);
    const uint16_t* r = static_cast<const uint16_t*>(a.router) + e * d.ld_router;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = lane * 8; k < H; k += 256) {
        const uint4 w = ld_row8<VEC>(r + k, H - k);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t >= nt) break;
            const uint4 v = ld_row8<VEC>(x + (t0 + t) * d.ldx + k, H - k);
            const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<T>(ww[i]), g = unpack2<T>(vv[i]);
                acc[t] = fmaf(f.x, g.x, acc[t]);
                acc[t] = fmaf(f.y, g.y, acc[t]);
            }
        }
    }
    float* z = reinterpret_cast<float*>(a.ws + a.w.logits);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
        if (lane == 0 && t < nt) z[(t0 + t) * d.E + e] = acc[t];
    }
}

// ------------------------------------------------------------------ experts
struct MoeShared {
    unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
    int off[kMoeMaxExperts];                  // first slot of each expert
    int active[kMoeMaxExperts];               // experts that have tokens
    int n_active;
    int warp_first[kMoeWarps], warp_last[kMoeWarps];  // output blocks that each warp adds to
    int last[2];                              // this CTA joins its first / last output block
    int gave_up;
    int slot_token[kMoeMaxTokens * kMoeMaxTopK];
    float slot_weight[kMoeMaxTokens * kMoeMaxTopK];
    short pick[kMoeMaxTokens * kMoeMaxTopK];
    float pick_weight[kMoeMaxTokens * kMoeMaxTopK];
};

// Order-preserving key of a logit; NaN below every number, 0 is free for "not there".
__device__ __forceinline__ uint32_t order_key(float z) {
    if (z != z) return 1u;
    const uint32_t b = __float_as_uint(z + 0.0f);  // -0 becomes +0: equal logits, equal keys
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Top-k of one token by a warp, PER logits a lane: writes pick[] and pick_weight[] at t * top_k.
template <int PER>
__device__ __forceinline__ void route_token(const MoeArgs& a, MoeShared& s, int t, int lane) {
    const int E = static_cast<int>(a.d.E), k = static_cast<int>(a.d.top_k);
    const float* z = reinterpret_cast<const float*>(a.ws + a.w.logits) + static_cast<int64_t>(t) * E;
    float v[PER];
    uint32_t key[PER];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < E ? __ldcg(z + e) : 0.0f;
        key[i] = e < E ? order_key(v[i]) : 0u;
        if (e < E) top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i * 32 + lane < E) sum += expf(v[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    float total = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
        float bv = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) best = key[i], at = i * 32 + lane, bv = v[i];
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == m ? static_cast<uint32_t>(at) : 0xFFFFu);
        const float p = expf(__shfl_sync(0xFFFFFFFFu, bv, e & 31) - top) / sum;
        total += p;
        if (lane == 0) {
            s.pick[t * k + j] = static_cast<short>(e);
            s.pick_weight[t * k + j] = p;
            atomicOr(&s.mask[e], 1ull << t);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (static_cast<uint32_t>(i * 32 + lane) == e) key[i] = 0u;
    }
    __syncwarp();
    if (a.d.normalize)
        for (int j = lane; j < k; j += 32) s.pick_weight[t * k + j] /= total;
}

// One warp, steps [s0, s1) of 64 elements: acc[16 rows x 8 NT columns] += W x^T.  w0, w1: this
// lane's two weight rows (null: zeros), xr: its token rows (padded), K valid elements of a weight row.
template <typename T, int ROWS, int NT>
__device__ __forceinline__ void mma_steps(const uint16_t* w0, const uint16_t* w1, const uint16_t* const (&xr)[NT],
                                          int s0, int s1, int K, int t4, float (&acc)[NT][4]) {
    constexpr int U = NT <= 2 ? 2 : 1;  // steps of loads in a batch (two batches in flight)
    Row16 wa[2][U], wb[2][U];
    const auto load = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64 + t4 * 16;
            const int n = s + u < s1 ? K - k : 0;
            wa[b][u] = ld_row16<ROWS>(w0 + k, w0 ? n : 0);
            wb[b][u] = ld_row16<ROWS>(w1 + k, w1 ? n : 0);
        }
    };
    const auto compute = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const int k = (s + u) * 64 + t4 * 16;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 xv = *reinterpret_cast<const uint4*>(xr[j] + k + 8 * i);
                    const uint32_t *p = wa[b][u].v + 4 * i, *q = wb[b][u].v + 4 * i;
                    mma16816<T>(acc[j], p[0], q[0], p[1], q[1], xv.x, xv.y);
                    mma16816<T>(acc[j], p[2], q[2], p[3], q[3], xv.z, xv.w);
                }
            }
        }
    };
    load(0, s0);
    for (int s = s0; s < s1; s += 2 * U) {
        load(1, s + U);
        compute(0, s);
        load(0, s + 2 * U);
        compute(1, s + U);
    }
}

// As mma_steps for n columns (1 to 8 NTMAX) of the slots at `off`: rows of `x` of xld elements, indexed
// by token (by_token) or by slot.
template <typename T, int ROWS, int NTMAX>
__device__ __forceinline__ void mma_cols(const MoeShared& s, const uint16_t* w0, const uint16_t* w1,
                                         const uint16_t* x, int64_t xld, bool by_token, int off, int n, int s0,
                                         int s1, int K, int lane, float (&acc)[NTMAX][4]) {
    const auto run = [&](auto tag) {
        constexpr int NT = decltype(tag)::value;
        const uint16_t* xr[NT];
        float c[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            // columns past the last read its row: their sums are not used
            const int slot = off + min(j * 8 + (lane >> 2), n - 1);
            xr[j] = x + (by_token ? s.slot_token[slot] : slot) * xld;
#pragma unroll
            for (int i = 0; i < 4; ++i) c[j][i] = 0.0f;
        }
        mma_steps<T, ROWS, NT>(w0, w1, xr, s0, s1, K, lane & 3, c);
#pragma unroll
        for (int j = 0; j < NTMAX; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = j < NT ? c[j < NT ? j : 0][i] : 0.0f;
    };
    if constexpr (NTMAX >= 8) {
        if (n > 32) return run(std::integral_constant<int, 8>{});
    }
    if constexpr (NTMAX >= 4) {
        if (n > 16) return run(std::integral_constant<int, 4>{});
    }
    if constexpr (NTMAX >= 2) {
        if (n > 8) return run(std::integral_constant<int, 2>{});
    }
    run(std::integral_constant<int, 1>{});
}

template <typename T, int ROWS, int NTMAX>
__global__ void __launch_bounds__(MT, 1) moe_experts_kernel(const MoeArgs a) {
    extern __shared__ __align__(16) char moe_smem[];
    MoeShared& s = *reinterpret_cast<MoeShared*>(moe_smem);
    float* tiles = reinterpret_cast<float*>(moe_smem + (sizeof(MoeShared) + 15) / 16 * 16);
    const gemm_moe_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok = static_cast<int>(d.T), E = static_cast<int>(d.E), top_k = static_cast<int>(d.top_k);
    const int G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);

    // ---------------------------------------------------------------- routing
    for (int e = threadIdx.x; e < E; e += MT) s.mask[e] = 0ull;
    if (threadIdx.x == 0) s.gave_up = 0;
    __syncthreads();
    for (int t = warp; t < tok; t += kMoeWarps) {
        if (E <= 64)
            route_token<2>(a, s, t, lane);
        else
            route_token<kMoeMaxExperts / 32>(a, s, t, lane);
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0, slots = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? __popcll(s.mask[e]) : 0;
            const unsigned has = __ballot_sync(0xFFFFFFFFu, c > 0);
            int pre = c;  // inclusive prefix sum of the counts
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, pre, o);
                if (lane >= o) pre += up;
            }
            if (e < E) s.off[e] = slots + pre - c;
            if (c > 0) s.active[n + __popc(has & ((1u << lane) - 1u))] = e;
            n += __popc(has);
            slots += __shfl_sync(0xFFFFFFFFu, pre, 31);
        }
        if (lane == 0) s.n_active = n;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tok * top_k; i += MT) {
        const int t = i / top_k, e = s.pick[i];
        const int slot = s.off[e] + __popcll(s.mask[e] & ((1ull << t) - 1ull));
        s.slot_token[slot] = t;
        s.slot_weight[slot] = s.pick_weight[i];
        if (cta == 0) {
            if (a.ids) a.ids[i] = e;
            if (a.weights) a.weights[i] = s.pick_weight[i];
        }
    }
    __syncthreads();
    const int A = s.n_active;

    // ---------------------------------------------------------------- up
    const uint16_t* xp = reinterpret_cast<const uint16_t*>(a.ws + a.w.x);
    T* h = reinterpret_cast<T*>(a.ws + a.w.h);
    const int g = lane >> 2, t4 = lane & 3;
    float* my_tile = tiles + warp * 2 * (16 * 8 * NTMAX);
    {
        const bool gated = d.act == GEMM_MOE_SWIGLU;
        const int per = gated ? 8 : 16;  // values of h per unit
        // (the host keeps these counts below 2^31)
        const int UB = static_cast<int>((d.I + per - 1) / per), U = UB * A;
        const int KS = static_cast<int>(a.w.hp / 64);
        const Share ctas(U, G);
        const int u_lo = ctas.lo(cta), total = (ctas.lo(cta + 1) - u_lo) * KS;
        const Share warps(total, kMoeWarps);
        const int lo = warps.lo(warp), hi = warps.lo(warp + 1);
        const uint16_t* w1 = static_cast<const uint16_t*>(a.w1);
        const auto finish = [&](int u, const float (&acc)[NTMAX][4]) {
            const int e = s.active[u / UB];
            const int i0 = u % UB * per;
            const int n = __popcll(s.mask[e]), off = s.off[e];
#pragma unroll
            for (int j = 0; j < NTMAX; ++j) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = j * 8 + t4 * 2 + c;
                    if (col >= n) continue;
                    T* row = h + (off + col) * a.w.ip;
                    const float v0 = acc[j][c], v1 = acc[j][2 + c];
                    if (gated) {
                        if (i0 + g < d.I) row[i0 + g] = cast16<T>(v0 / (1.0f + expf(-v0)) * v1);
                    } else {
                        if (i0 + g < d.I) row[i0 + g] = cast16<T>(moe_act(d.act, v0));
                        if (i0 + g + 8 < d.I) row[i0 + g + 8] = cast16<T>(moe_act(d.act, v1));
                    }
                }
            }
        };
        for (int cur = lo; cur < hi;) {
            const int u = u_lo + cur / KS;
            const int s0 = cur % KS, s1 = min(KS, s0 + hi - cur);
            const int e = s.active[u / UB];
            const int64_t i = u % UB * per + g;
            const uint16_t* base = w1 + e * d.stride_w1;
            const uint16_t* r0 = i < d.I ? base + i * d.ld_w1 : nullptr;
            const uint16_t* r1 = gated ? (r0 ? r0 + d.I * d.ld_w1 : nullptr)
                                       : (i + 8 < d.I ? base + (i + 8) * d.ld_w1 : nullptr);
            float acc[NTMAX][4];
            mma_cols<T, ROWS, NTMAX>(s, r0, r1, xp, a.w.hp, true, s.off[e], __popcll(s.mask[e]), s0, s1,
                                    static_cast<int>(d.H), lane, acc);
            if (s0 == 0 && s1 == KS) {
                finish(u, acc);
            } else {
                // a unit that began in an earlier warp goes to slot 0, one that goes on in a later
                // warp to slot 1
                float* slot = my_tile + (s0 > 0 ? 0 : 16 * 8 * NTMAX);
#pragma unroll
                for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) slot[(j * 4 + c) * 32 + lane] = acc[j][c];
            }
            cur += s1 - s0;
        }
        __syncthreads();
        // the warp in which a cut unit begins joins it
        if (lo < hi) {
            const int u = (hi - 1) / KS;
            if (u * KS >= lo && (u + 1) * KS > hi) {
                float acc[NTMAX][4];
#pragma unroll
                for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[j][c] = my_tile[16 * 8 * NTMAX + (j * 4 + c) * 32 + lane];
                for (int w = warp + 1; w < kMoeWarps; ++w) {
                    if (warps.lo(w) >= (u + 1) * KS || warps.lo(w) == warps.lo(w + 1)) break;
                    const float* slot = tiles + w * 2 * (16 * 8 * NTMAX);
#pragma unroll
                    for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[j][c] += slot[(j * 4 + c) * 32 + lane];
                }
                finish(u_lo + u, acc);
            }
        }
    }

    // ---------------------------------------------------------------- grid barrier
    // This warp's share of the down product is known already: its first weights are
    // asked into L2 while the barrier is waited for.
    const int OB = static_cast<int>((d.H + 15) / 16), V = OB * A;
    const int KS = static_cast<int>(a.w.ip / 64);
    const Share ctas(V, G);
    const int v_lo = ctas.lo(cta), v_hi = ctas.lo(cta + 1);
    const Share warps((v_hi - v_lo) * KS, kMoeWarps);
    const int lo = warps.lo(warp), hi = warps.lo(warp + 1);
    const uint16_t* w2 = static_cast<const uint16_t*>(a.w2);
    if (lo < hi) {
        const int v = v_lo + lo / KS, k = (lo % KS + t4) * 64;
        const int64_t o = v / A * 16 + g;
        const uint16_t* p = w2 + s.active[v % A] * d.stride_w2 + o * d.ld_w2 + k;
        if (k < d.I && o < d.H) prefetch_l2(p);
        if (k < d.I && o + 8 < d.H) prefetch_l2(p + 8 * d.ld_w2);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned* bar = reinterpret_cast<unsigned*>(a.ws + a.w.bar);
        __threadfence();
        if (!((d.flags & GEMM_FLAG_TEST_STALL) && cta == 0)) atomicAdd(bar, 1u);
        const uint64_t t0 = globaltimer_ns();
        while (ld_acquire_gpu(bar) < static_cast<unsigned>(G)) {
            if (globaltimer_ns() - t0 > a.timeout_ns) {
                atomicOr(a.status, DEVERR_TIMEOUT);
                s.gave_up = 1;
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
    if (s.gave_up) return;

    // ---------------------------------------------------------------- down
    const int ytile = 16 * tok;  // [row][token]
    float* yt = tiles + warp * 2 * ytile;
    for (int i = lane; i < 2 * ytile; i += 32) yt[i] = 0.0f;
    __syncwarp();
    const int first_ob = (v_lo + lo / KS) / A;
    if (lane == 0) {
        s.warp_first[warp] = first_ob;
        s.warp_last[warp] = lo < hi ? (v_lo + (hi - 1) / KS) / A : -1;
    }
    for (int cur = lo; cur < hi;) {
        const int v = v_lo + cur / KS;
        const int s0 = cur % KS, s1 = min(KS, s0 + hi - cur);
        const int ob = v / A;
        const int e = s.active[v - ob * A];
        const int64_t o = ob * 16 + g;
        const uint16_t* base = w2 + e * d.stride_w2;
        const uint16_t* r0 = o < d.H ? base + o * d.ld_w2 : nullptr;
        const uint16_t* r1 = o + 8 < d.H ? base + (o + 8) * d.ld_w2 : nullptr;
        const int n = __popcll(s.mask[e]), off = s.off[e];
        float acc[NTMAX][4];
        mma_cols<T, ROWS, NTMAX>(s, r0, r1, reinterpret_cast<const uint16_t*>(h), a.w.ip, false, off, n, s0, s1,
                                static_cast<int>(d.I), lane, acc);
        float* tile = yt + (ob == first_ob ? 0 : ytile);
#pragma unroll
        for (int j = 0; j < NTMAX; ++j) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = j * 8 + t4 * 2 + c;
                if (col >= n) continue;
                const int t = s.slot_token[off + col];
                const float wgt = s.slot_weight[off + col];
                tile[g * tok + t] += wgt * acc[j][c];
                tile[(g + 8) * tok + t] += wgt * acc[j][2 + c];
            }
        }
        __syncwarp();
        cur += s1 - s0;
    }
    __syncthreads();

    // Output blocks of this CTA: the sums of its warps, in order.
    T* y = static_cast<T*>(a.y);
    float* partial = reinterpret_cast<float*>(a.ws + a.w.partial);
    if (v_lo >= v_hi) return;
    const int ob_lo = v_lo / A, ob_hi = (v_hi - 1) / A;
    for (int i = threadIdx.x; i < (ob_hi - ob_lo + 1) * ytile; i += MT) {
        const int ob = ob_lo + i / ytile, el = i % ytile;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kMoeWarps; ++w)
            if (ob >= s.warp_first[w] && ob <= s.warp_last[w])
                sum += tiles[(w * 2 + (ob == s.warp_first[w] ? 0 : 1)) * ytile + el];
        if (ob * A >= v_lo && (ob + 1) * A <= v_hi) {
            const int o = ob * 16 + el / tok;
            if (o < d.H) y[(el % tok) * d.ldy + o] = cast16<T>(sum);
        } else {
            partial[(cta * 2 + (ob == ob_lo ? 0 : 1)) * ytile + el] = sum;
        }
    }
    // The first and the last block: whoever arrives last at a cut one joins it.
    if (ob_lo * A >= v_lo && (ob_hi + 1) * A <= v_hi) return;  // neither is cut
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2) {
        const int ob = threadIdx.x == 0 ? ob_lo : ob_hi;
        const bool whole = ob * A >= v_lo && (ob + 1) * A <= v_hi;
        int last = 0;
        if (!whole && (threadIdx.x == 0 || ob_hi != ob_lo)) {
            // blocks are cut between neighbours, none of which is empty
            const unsigned parts = ctas.owner(ob * A + A - 1) - ctas.owner(ob * A) + 1;
            unsigned* ctr = reinterpret_cast<unsigned*>(a.ws + a.w.counters);
            last = atomicAdd(ctr + ob, 1u) == parts - 1;
            __threadfence();
        }
        s.last[threadIdx.x] = last;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!s.last[k]) continue;
        const int ob = k == 0 ? ob_lo : ob_hi;
        const int c_lo = ctas.owner(ob * A), c_hi = ctas.owner(ob * A + A - 1);
        for (int el = threadIdx.x; el < ytile; el += MT) {
            float sum = 0.0f;
            // the first of them may have begun in an earlier block: then this one is its last
            for (int c = c_lo; c <= c_hi; ++c)
                sum += __ldcg(partial + (c * 2 + (c > c_lo || ctas.lo(c) >= ob * A ? 0 : 1)) * ytile + el);
            const int o = ob * 16 + el / tok;
            if (o < d.H) y[(el % tok) * d.ldy + o] = cast16<T>(sum);
        }
    }
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

template <typename T, int ROWS, int NTMAX>
cudaError_t launch_experts(const MoeArgs& a, int grid, cudaStream_t st) {
    auto k = moe_experts_kernel<T, ROWS, NTMAX>;
    const size_t smem = (sizeof(MoeShared) + 15) / 16 * 16 +
                        static_cast<size_t>(kMoeWarps) * 2 * 16 * 8 * NTMAX * sizeof(float);
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(MT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;  // the grid barrier needs every CTA resident
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T, int ROWS>
cudaError_t launch_t(const MoeArgs& a, int grid, cudaStream_t st) {
    const int64_t units = a.d.E * ((a.d.T + 3) / 4);
    const unsigned blocks = static_cast<unsigned>((units + RT / 32 - 1) / (RT / 32));
    // the router's rows and x take vector loads on their own terms
    const bool rvec = reinterpret_cast<uintptr_t>(a.router) % 16 == 0 && a.d.ld_router % 8 == 0 &&
                      reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.d.ldx % 8 == 0 && a.d.H % 8 == 0;
    if (rvec)
        moe_router_kernel<T, true><<<blocks, RT, 0, st>>>(a);
    else
        moe_router_kernel<T, false><<<blocks, RT, 0, st>>>(a);
    cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return ce;
    // groups of 8 tokens that one expert can be given: 1, 2, 4 or 8
    if (a.d.T <= 8) return launch_experts<T, ROWS, 1>(a, grid, st);
    if (a.d.T <= 16) return launch_experts<T, ROWS, 2>(a, grid, st);
    if (a.d.T <= 32) return launch_experts<T, ROWS, 4>(a, grid, st);
    return launch_experts<T, ROWS, 8>(a, grid, st);
}

}  // namespace

MoeWorkspace moe_workspace(const gemm_moe_desc_t& d, int grid) {
    MoeWorkspace w{};
    w.hp = round_up(d.H, 64);
    w.ip = round_up(d.I, 64);
    w.bar = 0;
    w.counters = 256;
    w.logits = w.counters + round_up((d.H + 15) / 16 * 4, 256);
    w.x = w.logits + round_up(d.T * d.E * 4, 256);
    w.h = w.x + round_up(d.T * w.hp * 2, 256);
    w.partial = w.h + round_up(d.T * d.top_k * w.ip * 2, 256);
    w.bytes = w.partial + static_cast<int64_t>(grid) * 2 * 16 * d.T * 4;
    return w;
}

cudaError_t launch_moe(const MoeArgs& a, int grid, cudaStream_t st) {
    const auto all = [&](int64_t n) {  // every row on n elements, rows a multiple of n long
        return reinterpret_cast<uintptr_t>(a.w1) % (2 * n) == 0 && reinterpret_cast<uintptr_t>(a.w2) % (2 * n) == 0 &&
               a.d.ld_w1 % n == 0 && a.d.ld_w2 % n == 0 && a.d.stride_w1 % n == 0 && a.d.stride_w2 % n == 0 &&
               a.d.H % n == 0 && a.d.I % n == 0;
    };
    const bool f16 = a.d.dtype == GEMM_F16;
    if (all(16)) return f16 ? launch_t<__half, ROWS_32>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_32>(a, grid, st);
    if (all(8)) return f16 ? launch_t<__half, ROWS_16>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_16>(a, grid, st);
    return f16 ? launch_t<__half, ROWS_ANY>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_ANY>(a, grid, st);
}

}  // namespace g13
