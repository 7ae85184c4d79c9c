// moe_kernel.cuh -- a mixture-of-experts layer for a few tokens (1 to 64):
//
//   z = x Wr^T;  p = softmax(z) over all experts;  the top_k largest z (ties: the
//   lowest index) with weights p, or p divided by their sum;
//   y = sum_j weight_j  W2[e_j] act(W1[e_j] x)
//   act: GELU or ReLU of I rows, or SwiGLU: silu(gate) * up, gate = rows 0..I-1 of
//   W1[e], up = rows I..2I-1
//
// or with experts and weights of each token that were chosen beforehand, instead of the first two lines (GIVEN: kernels of
// their own; with both in one, asked for while it runs, the layer with a router took 116 us instead of 112 below).
//
// A few tokens leave two products per weight byte and token: reading the chosen
// experts' weights once is the cost, so everything is laid out to keep those
// loads in flight.  Two kernels:
//
//   router   z in FP32 (a CTA per two experts and four tokens); copies x into rows
//            padded to 64 elements; clears the counters of the second kernel
//   experts  one CTA of 16 warps per SM, cooperative.  Every CTA works out the
//            routing for itself from z (softmax, top-k by warp-wide maximum
//            reductions, a 64-bit mask of tokens per expert), which is cheaper than
//            another trip through memory.  Then the two products, with one grid
//            barrier between them:
//     up     work units of 16 weight rows of a chosen expert (SwiGLU: 8 gate rows
//            and their 8 up rows, so one thread holds both factors) x 64-element
//            steps along H.  A CTA takes an equal share of the units' costs; its warps take
//            whole units in turn, and equal shares of the steps of those left over,
//            joined through shared memory in warp order.
//     down   units (64 output columns, chosen expert), column block major; CTAs, and
//            their teams of four warps, take equal shares of all units' steps; each
//            warp adds weight * product to its own tile of the output in shared
//            memory.  A block cut between CTAs leaves partial sums in the workspace,
//            and the CTA that arrives last adds them in CTA order.
//   No sum depends on timing.
//
// Weights go from global memory straight into registers, two batches ahead.  (Through a
// ring in shared memory, cp.async per warp, they took 118 us where this took 113 with 16 tokens,
// and 600 against 445 with 64, h in one part: the ring's space is what L1 keeps the tokens' values in.)  Rows
// that are not 16-byte aligned are loaded as the granules that hold them and shifted.
//
// Measured (bytes of the chosen experts over time): 16 tokens, 64 experts of 2048 x 1024:
// 110 us, 5.7 TB/s (0.85 of a copy's rate); 64 tokens, 64 experts of 4096 x 1536: 467 us,
// 5.2 TB/s (the tokens' values take half of what the SMs read; where an expert has 32
// tokens or more they take most of it, and 2.5 TB/s remain); one token, 2 of 8
// experts of 768 x 3072: 16 us, of which 3 are bytes and the rest a chain of two
// kernels, the routing, the barrier and the join, each a trip or two to L2.  (Blocks of
// 16 columns instead of 64 in the down product cut fewer of them between CTAs and
// still took 17 us: sixteen teams' sums are slower to add than four's.)
//
// Products: mma.sync m16n8k16, weights as the 16 rows and a group of 8 tokens as
// the columns.  The order of k within a step is free as long as both operands share
// it, so a thread takes 16 consecutive values of a row (four MMAs' worth) as its
// fragments.  (tcgen05 would need a 128-row tile and TMEM round trips, to do
// arithmetic that is far from the bound.)  FP32 accumulation; h = act(...) goes into the
// second product, whose operands are 16-bit, as two numbers of that type, its rounding and
// the rest.  (Rounded once, it made the output's error 1.4 times that of the output's own
// rounding, and the layers took 112, 452 and 16 us.)
#pragma once
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
constexpr int kMoeTeams = kMoeWarps / 4;  // down product: teams of four warps
constexpr int RT = 256;              // threads per router CTA
constexpr int kMaxDevices = 64;

// h is held in two parts, its rounding and the rest.  FP16 has a second such array, in units of 2^16, for the
// values beyond its range (the router clears it; the second product reads it only where one exists).
constexpr float kMoeBigUnit = 65536.0f, kMoeBigFrom = 65520.0f;  // (less rounds to 65504)
template <typename T>
constexpr bool kMoeBig = std::is_same<T, __half>::value;

// A 16-byte piece of a row.  (Two loads meet in most 32-byte sectors: without room in L1 the second
// would fetch it again; 132 us instead of 144 with 16 tokens and unaligned rows, 525 instead of 659
// with 64, h still in one part.)
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::evict_first.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

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
// How the rows of a weight lie: all on 32 bytes with lengths a multiple of 16 elements, all
// on 16 bytes with multiples of 8, or anyhow.
enum Rows { ROWS_32 = 0, ROWS_16 = 1, ROWS_ANY = 2 };

// Sixteen values of an aligned row, n of which exist (n <= 0: none; else, with the row's
// length, 8 or 16 at least).
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
        const uint4 a = ld_row8<true>(p, n), b = ld_row8<true>(p + 8, n - 8);
        r = Row16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return r;
}

// Sixteen values of a row that lies anyhow, as they are loaded: the three 16-byte granules
// that hold them (two, where they are aligned), to be shifted when they are used.
struct Raw16 {
    uint32_t v[12];
};
// (`on` false: nothing is loaded and r keeps what it holds.  The predicate sits inside the
// assembly: a branch, or zeros for the other case, cost the loop its schedule.)
__device__ __forceinline__ void ld_raw16(Raw16& r, const char* p, bool on, unsigned o) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@p ld.global.nc.L1::evict_first.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(r.v[4 * i]), "+r"(r.v[4 * i + 1]), "+r"(r.v[4 * i + 2]), "+r"(r.v[4 * i + 3])
            : "l"(p + 16 * i), "r"(static_cast<int>(on && (i < 2 || o != 0))));
}
// The values themselves; o: their offset in bytes in the first granule.
__device__ __forceinline__ void use_raw16(const Raw16& r, unsigned o, uint32_t (&w)[8]) {
    uint32_t v[12];
#pragma unroll
    for (int i = 0; i < 12; ++i) v[i] = r.v[i];
#pragma unroll
    for (int i = 0; i < 10; ++i) v[i] = o & 8 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) v[i] = o & 4 ? v[i + 1] : v[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], (o & 2) * 8);
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

__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

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
__device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// A number in two parts (an infinity, or NaN, in the first alone), the second `step` elements on.
template <typename T>
__device__ __forceinline__ void two_parts(T* p, int64_t step, float v) {
    const T hi = cast16<T>(v);
    const float f = as_float(hi);
    p[0] = hi;
    p[step] = cast16<T>(fabsf(f) < INFINITY ? v - f : 0.0f);
}

// ------------------------------------------------------------------ router
// A CTA takes two experts and four tokens; its threads take 8 elements of H each, so that
// everything a CTA reads is in flight at once.
constexpr int RE = 2, RTOK = 4;

template <typename T, bool VEC, bool GIVEN>
__global__ void __launch_bounds__(RT) moe_router_kernel(const MoeArgs a) {
    griddep_launch();  // the experts' kernel may take its place; it waits for this one's results
    griddep_wait();    // what came before has written its inputs, and is done with the workspace
    __shared__ float sums[RT / 32][RE * RTOK];
    const gemm_moe_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = static_cast<int>(d.E), H = static_cast<int>(d.H), tok = static_cast<int>(d.T);
    const int groups = (E + RE - 1) / RE;
    const int e0 = static_cast<int>(blockIdx.x) % groups * RE, t0 = static_cast<int>(blockIdx.x) / groups * RTOK;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* r = static_cast<const uint16_t*>(a.router);
    float acc[RE][RTOK] = {};
    for (int k = GIVEN ? H : threadIdx.x * 8; k < H; k += RT * 8) {
        uint4 w[RE], v[RTOK];
#pragma unroll
        for (int e = 0; e < RE; ++e) w[e] = ld_row8<VEC>(r + (e0 + e) * d.ld_router + k, e0 + e < E ? H - k : 0);
#pragma unroll
        for (int t = 0; t < RTOK; ++t) v[t] = ld_row8<VEC>(x + (t0 + t) * d.ldx + k, t0 + t < tok ? H - k : 0);
#pragma unroll
        for (int e = 0; e < RE; ++e)
#pragma unroll
            for (int t = 0; t < RTOK; ++t) {
                const uint32_t ww[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
                const uint32_t vv[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<T>(ww[i]), g = unpack2<T>(vv[i]);
                    acc[e][t] = fmaf(f.x, g.x, acc[e][t]);
                    acc[e][t] = fmaf(f.y, g.y, acc[e][t]);
                }
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < RE * RTOK; ++i)
            acc[i / RTOK][i % RTOK] += __shfl_xor_sync(0xFFFFFFFFu, acc[i / RTOK][i % RTOK], o);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < RE * RTOK; ++i) sums[warp][i] = acc[i / RTOK][i % RTOK];
    __syncthreads();
    const int e = e0 + static_cast<int>(threadIdx.x) / RTOK, t = t0 + static_cast<int>(threadIdx.x) % RTOK;
    if (threadIdx.x < RE * RTOK && e < E && t < tok && !GIVEN) {
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < RT / 32; ++w) z += sums[w][threadIdx.x];
        reinterpret_cast<float*>(a.ws + a.w.logits)[t * E + e] = z;
    }

    // the counters, the padded copy of x, and the padding of h (which the up product does not write)
    // (every count here stays below 2^31; 64-bit divisions would cost microseconds)
    const int tid = static_cast<int>(blockIdx.x) * RT + threadIdx.x;
    const int nthreads = static_cast<int>(gridDim.x) * RT;
    unsigned* ctr = reinterpret_cast<unsigned*>(a.ws + a.w.bar);
    const int n_ctr = static_cast<int>((a.w.logits - a.w.bar) / 4);
    for (int i = tid; i < n_ctr; i += nthreads) ctr[i] = 0u;
    uint16_t* xp = reinterpret_cast<uint16_t*>(a.ws + a.w.x);
    const int hp8 = static_cast<int>(a.w.hp / 8);
    for (int i = tid; i < tok * hp8; i += nthreads) {
        const int row = i / hp8, k = (i - row * hp8) * 8;
        reinterpret_cast<uint4*>(xp)[i] = ld_row8<VEC>(x + row * d.ldx + k, H - k);
    }
    uint16_t* h = reinterpret_cast<uint16_t*>(a.ws + a.w.h);
    const int pad = static_cast<int>(a.w.ip - d.I), parts = static_cast<int>(d.T * d.top_k) * 2;
    for (int i = tid; i < parts * pad; i += nthreads)  // both parts of each h
        h[static_cast<int64_t>(i / pad) * a.w.ip + d.I + i % pad] = 0;
    if constexpr (kMoeBig<T>) {
        uint4* big = reinterpret_cast<uint4*>(h + parts * a.w.ip);
        const int64_t n = parts * (a.w.ip / 8);
        for (int64_t i = tid; i < n; i += nthreads) big[i] = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ experts
struct MoeShared {
    unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
    short off[kMoeMaxExperts];                // first slot of each expert
    short active[kMoeMaxExperts];             // experts that have tokens
    short cost[kMoeMaxExperts];               // of each of them: the unit costs of those before it
    float slot_weight[kMoeMaxTokens * kMoeMaxTopK];
    uint8_t slot_token[kMoeMaxTokens * kMoeMaxTopK];
    int n_active, all_cost;
    int u_lo, u_hi;  // this CTA's units of the up product
    int team_first[kMoeTeams], team_last[kMoeTeams];  // output blocks that each team adds to
    int last[2];                              // this CTA joins its first / last output block
    int gave_up;
    int big;  // a value of h lies beyond FP16: one that this CTA wrote, after the barrier one that any wrote
};
// While the routing is worked out, each token's choice lies where the tiles of sums are later.
struct MoePicks {
    float weight[kMoeMaxTokens * kMoeMaxTopK];
    short expert[kMoeMaxTokens * kMoeMaxTopK];
};

// Time of a unit of the up product by its expert's tokens (the more columns, the more of its time goes to
// the tokens' values; ratios as measured with every expert alike): the CTAs' shares are equal in this.
// Shares of equally many units gave all units of a busy expert to two or three CTAs, and every other one
// waited for them at the barrier: 64 tokens, 8 of 64 experts of 4096 x 1536, one of which has 17: 630 us
// instead of 482; none of which has more than 16: 486 instead of 467.
__device__ __forceinline__ int unit_cost(int n) {
    return n <= 8 ? 5 : n <= 16 ? 6 : n <= 32 ? 10 : 15;
}

// Order-preserving key of a logit; NaN below every number, 0 is free for "not there".
__device__ __forceinline__ uint32_t order_key(float z) {
    if (z != z) return 1u;
    const uint32_t b = __float_as_uint(z + 0.0f);  // -0 becomes +0: equal logits, equal keys
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The logit that a key stands for (-0 as +0).
__device__ __forceinline__ float key_value(uint32_t key) {
    if (key == 1u) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Top-k of N tokens t0, t0 + step, ... (those below `tok`) by a warp, PER logits a lane:
// writes its picks at t * top_k.  A round finds the largest key, then
// the lowest index that has it; the tokens' rounds are independent and overlap.
template <int PER, int N>
__device__ __forceinline__ void route_tokens(const MoeArgs& a, MoeShared& s, MoePicks& picks, int t0, int step, int tok, int lane) {
    const int E = static_cast<int>(a.d.E), k = static_cast<int>(a.d.top_k);
    const float* z = reinterpret_cast<const float*>(a.ws + a.w.logits);
    uint32_t key[N][PER];
    float top[N], sum[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane, t = min(t0 + n * step, tok - 1);
            key[n][i] = e < E ? order_key(__ldcg(z + t * E + e)) : 0u;
        }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = max(m, key[n][i]);
        top[n] = key_value(__reduce_max_sync(0xFFFFFFFFu, m));  // (NaN only if every logit is NaN)
        sum[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane < E) sum[n] += expf(key_value(key[n][i]) - top[n]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) sum[n] += __shfl_xor_sync(0xFFFFFFFFu, sum[n], o);
    // lane j keeps pick j
    uint32_t my_key[N], my_e[N];
#pragma unroll
    for (int n = 0; n < N; ++n) my_key[n] = 1u, my_e[n] = 0u;
    for (int j = 0; j < k; ++j) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) m = max(m, key[n][i]);
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            uint32_t e = 0xFFFFu;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[n][i] == m) e = i * 32 + lane;
            e = __reduce_min_sync(0xFFFFFFFFu, e);
            if (lane == j) my_key[n] = m, my_e[n] = e;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i * 32 + lane == e) key[n][i] = 0u;
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float p = lane < k ? expf(key_value(my_key[n]) - top[n]) / sum[n] : 0.0f;
        if (a.d.normalize) {
            float total = p;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
            p /= total;
        }
        const int t = t0 + n * step;
        if (lane < k && t < tok) {
            picks.expert[t * k + lane] = static_cast<short>(my_e[n]);
            picks.weight[t * k + lane] = p;
            atomicOr(&s.mask[my_e[n]], 1ull << t);
        }
    }
}

// The choice made beforehand, a warp's tokens t0, t0 + step, ...: ids outside 0 .. E - 1 take no part (expert -1),
// and an expert that a token names twice is one pick with the sum of the weights.
__device__ __forceinline__ void take_given(const MoeArgs& a, MoeShared& s, MoePicks& picks, int t0, int step, int tok, int lane) {
    const int E = static_cast<int>(a.d.E), k = static_cast<int>(a.d.top_k);
    for (int t = t0; t < tok; t += step) {
        int e = lane < k ? __ldg(a.given_ids + t * k + lane) : -1;
        const float w = lane < k ? __ldg(a.given_weights + t * k + lane) : 0.0f;
        if (e < 0 || e >= E) e = -1;
        float sum = 0.0f;
        bool first = true;
        for (int j = 0; j < k; ++j) {
            const int o = __shfl_sync(0xFFFFFFFFu, e, j);
            const float ow = __shfl_sync(0xFFFFFFFFu, w, j);
            if (o == e) {
                sum += ow;
                first = first && j >= lane;
            }
        }
        if (!first) e = -1;
        if (lane < k) {
            picks.expert[t * k + lane] = static_cast<short>(e);
            picks.weight[t * k + lane] = sum;
            if (e >= 0) atomicOr(&s.mask[e], 1ull << t);
        }
    }
}

// The tokens of a unit's columns: this lane's rows (padded to whole steps of 128 bytes).  Up to
// 16 columns as pointers, read in 16-byte pieces; more as 32-bit offsets in steps, read in
// 32-byte pieces, which leaves registers (64 tokens on 8 of 16 experts each, 4096 x 1536: 237 us
// instead of 266; with few columns the address arithmetic stands before every load: 489 us
// instead of 452 with 64 tokens on 8 of 64 experts; h still in one part and shares of equally many units).
template <int NT>
struct Columns {
    static constexpr bool FEW = NT <= 2;
    const uint16_t* base;
    const uint16_t* ptr[FEW ? NT : 1];
    uint32_t row[FEW ? 1 : NT];
    __device__ __forceinline__ void set(int j, uint32_t first_step) {
        if constexpr (FEW)
            ptr[j] = base + static_cast<uint64_t>(first_step) * 64;
        else
            row[j] = first_step;
    }
};
// acc[16 rows x 8 NT columns] += 16 values of rows g and g + 8 (p, q) times the tokens' values of step s
// (from L1 or L2; asking for them a step ahead took registers from the weights and was slower).  PARTS = 2:
// and times their second parts, KS steps further on.
template <typename T, int NT, int NTMAX, int PARTS>
__device__ __forceinline__ void mma_step(const uint32_t (&p)[8], const uint32_t (&q)[8], const Columns<NT>& x, int s,
                                         int KS, int t4, float (&acc)[NTMAX][4]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            const int k = (s + part * KS) * 64 + t4 * 16;
            if constexpr (Columns<NT>::FEW) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(x.ptr[j] + k + 8 * i);
                    mma16816<T>(acc[j], p[4 * i], q[4 * i], p[4 * i + 1], q[4 * i + 1], v.x, v.y);
                    mma16816<T>(acc[j], p[4 * i + 2], q[4 * i + 2], p[4 * i + 3], q[4 * i + 3], v.z, v.w);
                }
            } else {
                const ulonglong4_32a v =
                    *reinterpret_cast<const ulonglong4_32a*>(x.base + static_cast<uint64_t>(x.row[j]) * 64 + k);
                const unsigned long long w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma16816<T>(acc[j], p[2 * i], q[2 * i], p[2 * i + 1], q[2 * i + 1], static_cast<uint32_t>(w[i]),
                                static_cast<uint32_t>(w[i] >> 32));
            }
        }
    }
}

// One warp, steps [s0, s1) of a unit whose rows lie anyhow.  w0, w1: this lane's two weight
// rows, x: its token rows, K elements of a weight row.
template <typename T, int NT, int NTMAX, int PARTS>
__device__ __forceinline__ void steps_any(const uint16_t* w0, const uint16_t* w1, const Columns<NT>& x,
                                          int s0, int s1, int K, int KS, int t4, float (&acc)[NTMAX][4]) {
    const int sf = min(s1, K / 64);  // steps before it are whole
    w0 += t4 * 16;
    w1 += t4 * 16;
    const unsigned o0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(w0) & 15);
    const unsigned o1 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(w1) & 15);
    const char* p0 = reinterpret_cast<const char*>(w0) - o0;
    const char* p1 = reinterpret_cast<const char*>(w1) - o1;
    Raw16 ra[2] = {}, rb[2] = {};
    const auto load = [&](int b, int s) {
        ld_raw16(ra[b], p0 + s * 128, s < sf, o0);
        ld_raw16(rb[b], p1 + s * 128, s < sf, o1);
    };
    const auto compute = [&](int b, int s) {
        if (s >= sf) return;
        uint32_t p[8], q[8];
        use_raw16(ra[b], o0, p);
        use_raw16(rb[b], o1, q);
        mma_step<T, NT, NTMAX, PARTS>(p, q, x, s, KS, t4, acc);
    };
    load(0, s0);
    for (int s = s0; s < sf; s += 2) {
        load(1, s + 1);
        compute(0, s);
        load(0, s + 2);
        compute(1, s + 1);
    }
    if (sf < s1) {  // the row's end
        const int k = sf * 64, n = K - k - t4 * 16;
        uint32_t p[8], q[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = ld_row8<false>(w0 + k + 8 * i, n - 8 * i);
            const uint4 b = ld_row8<false>(w1 + k + 8 * i, n - 8 * i);
            p[4 * i] = a.x, p[4 * i + 1] = a.y, p[4 * i + 2] = a.z, p[4 * i + 3] = a.w;
            q[4 * i] = b.x, q[4 * i + 1] = b.y, q[4 * i + 2] = b.z, q[4 * i + 3] = b.w;
        }
        mma_step<T, NT, NTMAX, PARTS>(p, q, x, sf, KS, t4, acc);
    }
}

// The same for rows that all lie on 16 bytes (ROWS_16) or 32 (ROWS_32) and are a multiple of
// that long: two batches of U steps in flight in registers, 64 KB per SM and batch at U = 2.  (Down, with
// one group of tokens, U = 1: one token 15.7 us instead of 16.2, 16 tokens 114 instead of 116; up, or with
// two groups, it is the slower one: 16 tokens 118 instead of 116, 64 tokens 498 instead of 486, at the time.)
template <typename T, int ROWS, int NT, int NTMAX, int PARTS>
__device__ __forceinline__ void steps_aligned(const uint16_t* w0, const uint16_t* w1, const Columns<NT>& x,
                                              int s0, int s1, int K, int KS, int t4, float (&acc)[NTMAX][4]) {
    constexpr int U = NT == 2 || (NT == 1 && PARTS == 1) ? 2 : 1;
    Row16 wa[2][U], wb[2][U];
    const auto load = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64 + t4 * 16;
            const int n = s + u < s1 ? K - k : 0;
            wa[b][u] = ld_row16<ROWS>(w0 + k, n);
            wb[b][u] = ld_row16<ROWS>(w1 + k, n);
        }
    };
    const auto compute = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            mma_step<T, NT, NTMAX, PARTS>(wa[b][u].v, wb[b][u].v, x, s + u, KS, t4, acc);
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

template <typename T, int ROWS, int NT, int NTMAX, int PARTS>
__device__ __forceinline__ void steps(const uint16_t* w0, const uint16_t* w1, const Columns<NT>& x, int s0,
                                      int s1, int K, int KS, int t4, float (&acc)[NTMAX][4]) {
    if constexpr (ROWS == ROWS_ANY)
        steps_any<T, NT, NTMAX, PARTS>(w0, w1, x, s0, s1, K, KS, t4, acc);
    else
        steps_aligned<T, ROWS, NT, NTMAX, PARTS>(w0, w1, x, s0, s1, K, KS, t4, acc);
}

// Runs f with the least of 1, 2, 4, 8 (at most NTMAX) groups of 8 columns that hold n.
template <int NTMAX, typename F>
__device__ __forceinline__ void with_groups(int n, const F& f) {
    if constexpr (NTMAX >= 8) {
        if (n > 32) return f(std::integral_constant<int, 8>{});
    }
    if constexpr (NTMAX >= 4) {
        if (n > 16) return f(std::integral_constant<int, 4>{});
    }
    if constexpr (NTMAX >= 2) {
        if (n > 8) return f(std::integral_constant<int, 2>{});
    }
    f(std::integral_constant<int, 1>{});
}

template <int NTMAX>
constexpr int kMoeTileBytes = 2 * kMoeWarps * 16 * 8 * NTMAX * 4;
template <int NTMAX>
constexpr int kMoeSmem = (static_cast<int>(sizeof(MoeShared)) + 127) / 128 * 128 +
                         (kMoeTileBytes<NTMAX> > static_cast<int>(sizeof(MoePicks))
                              ? kMoeTileBytes<NTMAX>
                              : static_cast<int>(sizeof(MoePicks)));

// Moves this thread's values of h that lie beyond FP16, of a unit's sums, to their own array.  Out of line, as
// below: in the unit's own code it cost one token 0.9 us of 16.6 (instructions to fetch) and 16 tokens on
// unaligned rows 5 %; so it is 0.5 us and 3 %, the clearing of the array included.
template <typename T, int NTMAX>
__device__ __noinline__ void put_big(const MoeArgs& a, const float (&acc)[NTMAX][4], int e, int i0) {
    extern __shared__ __align__(128) uint8_t moe_smem[];
    MoeShared& s = *reinterpret_cast<MoeShared*>(moe_smem);
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, n = __popcll(s.mask[e]);
    const bool gated = a.d.act == GEMM_MOE_SWIGLU;
    T* h = reinterpret_cast<T*>(a.ws + a.w.h);
    for (int col = t4 * 2; col < n; col += col & 1 ? 7 : 1)
        for (int r = 0; r < (gated ? 1 : 2); ++r) {
            const float* v = &acc[col >> 3][col & 1];
            const float y = gated ? swiglu(v[0], v[2]) : moe_act(a.d.act, v[2 * r]);
            if (i0 + g + 8 * r >= a.d.I || !(fabsf(y) >= kMoeBigFrom && fabsf(y) < INFINITY)) continue;
            T* p = h + (s.off[e] + col) * 2 * a.w.ip + i0 + g + 8 * r;
            two_parts(p, a.w.ip, 0.0f);
            two_parts(p + a.d.T * a.d.top_k * 2 * a.w.ip, a.w.ip, y * (1.0f / kMoeBigUnit));
            s.big = 1;
        }
}

// What the values of h beyond FP16 give to a warp's sums of the down product: elementwise, for the columns that
// have any.  Out of line, and with nothing handed over that the kernel would have to keep in registers, since few layers
// ever come here.  (The products with this array by the loop that takes the others cost every FP16 layer of 64
// tokens 8 %, this function with the loop's variables as arguments 4 %.  Where most of h lies beyond FP16 a layer
// takes 2 to 8 times as long: 16 tokens, 64 experts of 2048 x 1024, 400 us instead of 111.)
template <typename T, int NTMAX>
__device__ __noinline__ void add_big(const MoeArgs& a) {
    extern __shared__ __align__(128) uint8_t moe_smem[];
    const MoeShared& s = *reinterpret_cast<const MoeShared*>(moe_smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & 3, team = warp >> 2;
    const int cta = static_cast<int>(blockIdx.x), tok = static_cast<int>(a.d.T), A = s.n_active;
    const int H = static_cast<int>(a.d.H), I = static_cast<int>(a.d.I), KS = static_cast<int>(a.w.ip / 64);
    const Share ctas((H + kMoeBlock - 1) / kMoeBlock * A * KS, static_cast<int>(gridDim.x));
    const int c_lo = ctas.lo(cta);
    const Share teams(ctas.lo(cta + 1) - c_lo, kMoeTeams);
    const int lo = c_lo + teams.lo(team), hi = c_lo + teams.lo(team + 1);
    float* yt = reinterpret_cast<float*>(moe_smem + (sizeof(MoeShared) + 127) / 128 * 128) + warp * 2 * 16 * 8 * NTMAX;
    float* flushed = reinterpret_cast<float*>(a.ws + a.w.flushed) + ((cta * kMoeTeams + team) * kMoeBlock + sub * 16) * tok;
    const T* h = reinterpret_cast<const T*>(a.ws + a.w.h) + a.d.T * a.d.top_k * 2 * a.w.ip;
    for (int cur = lo; cur < hi;) {
        const int v = cur / KS, s0 = cur % KS, s1 = min(KS, s0 + hi - cur);
        const int ob = v / A, e = s.active[v - ob * A], n = __popcll(s.mask[e]);
        float* sums = ob == (hi - 1) / KS / A ? yt : flushed;
        const int k0 = s0 * 64 + lane, k1 = min(s1 * 64, I);
        for (int c = 0; c < n; ++c) {
            const int slot = s.off[e] + c;
            const T* b = h + slot * 2 * a.w.ip;
            bool any = false;
            for (int k = k0; k < k1; k += 32) any = any || as_float(b[k]) != 0.0f;
            if (!__any_sync(0xFFFFFFFFu, any)) continue;
            for (int r = 0; r < 16; ++r) {
                const T* row = static_cast<const T*>(a.w2) + e * a.d.stride_w2 +
                               min(ob * kMoeBlock + sub * 16 + r, H - 1) * a.d.ld_w2;
                float sum = 0.0f;
                for (int k = k0; k < k1; k += 32) sum = fmaf(as_float(row[k]), as_float(b[k]) + as_float(b[a.w.ip + k]), sum);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                if (lane == 0) sums[r * tok + s.slot_token[slot]] += s.slot_weight[slot] * kMoeBigUnit * sum;
            }
        }
        __syncwarp();
        cur += s1 - s0;
    }
}

template <typename T, int ROWS, int NTMAX, bool GIVEN>
__global__ void __launch_bounds__(MT, 1) moe_experts_kernel(const __grid_constant__ MoeArgs a) {
    constexpr int TILE = 16 * 8 * NTMAX;  // a warp's tile of sums
    extern __shared__ __align__(128) uint8_t moe_smem[];
    MoeShared& s = *reinterpret_cast<MoeShared*>(moe_smem);
    float* tiles = reinterpret_cast<float*>(moe_smem + (sizeof(MoeShared) + 127) / 128 * 128);
    MoePicks& picks = *reinterpret_cast<MoePicks*>(tiles);
    const gemm_moe_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok = static_cast<int>(d.T), E = static_cast<int>(d.E), top_k = static_cast<int>(d.top_k);
    const int G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);

    // ---------------------------------------------------------------- routing
    for (int e = threadIdx.x; e < E; e += MT) s.mask[e] = 0ull;
    if (threadIdx.x == 0) s.gave_up = s.big = 0;
    griddep_wait();  // the router's results
    __syncthreads();
    static_assert(kMoeMaxTopK <= 32, "a lane for each pick");
    if constexpr (GIVEN) {
        take_given(a, s, picks, warp, kMoeWarps, tok, lane);
    } else if (E > 64) {
        for (int t = warp; t < tok; t += kMoeWarps)
            route_tokens<kMoeMaxExperts / 32, 1>(a, s, picks, t, kMoeWarps, tok, lane);
    } else if (tok > 2 * kMoeWarps) {
        for (int t = warp; t < tok; t += 4 * kMoeWarps) route_tokens<2, 4>(a, s, picks, t, kMoeWarps, tok, lane);
    } else if (tok > kMoeWarps) {
        route_tokens<2, 2>(a, s, picks, warp, kMoeWarps, tok, lane);
    } else if (warp < tok) {
        route_tokens<2, 1>(a, s, picks, warp, kMoeWarps, tok, lane);
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0, slots = 0;  // (with the costs in the high 16 bits, as in the sums below)
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? __popcll(s.mask[e]) : 0;
            const unsigned has = __ballot_sync(0xFFFFFFFFu, c > 0);
            const int both = c + (c > 0 ? unit_cost(c) << 16 : 0);
            int pre = both;  // inclusive prefix sums of the counts and the costs
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, pre, o);
                if (lane >= o) pre += up;
            }
            const int before = slots + pre - both;
            if (e < E) s.off[e] = static_cast<short>(before & 0xFFFF);
            if (c > 0) {
                const int i = n + __popc(has & ((1u << lane) - 1u));
                s.active[i] = static_cast<short>(e);
                s.cost[i] = static_cast<short>(before >> 16);
            }
            n += __popc(has);
            slots += __shfl_sync(0xFFFFFFFFu, pre, 31);
        }
        if (lane == 0) s.n_active = n, s.all_cost = slots >> 16;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tok * top_k; i += MT) {
        const int t = i / top_k, e = picks.expert[i];
        if (GIVEN && e < 0) continue;
        const int slot = s.off[e] + __popcll(s.mask[e] & ((1ull << t) - 1ull));
        s.slot_token[slot] = static_cast<uint8_t>(t);
        s.slot_weight[slot] = picks.weight[i];
        if (cta == 0) {
            if (a.ids) a.ids[i] = e;
            if (a.weights) a.weights[i] = picks.weight[i];
        }
    }
    const int A = s.n_active;
    if (GIVEN && A == 0) {  // (of choices made beforehand) no token has an expert
        for (int64_t i = cta * MT + static_cast<int>(threadIdx.x); i < tok * d.H; i += static_cast<int64_t>(G) * MT)
            static_cast<T*>(a.y)[i / d.H * d.ldy + i % d.H] = cast16<T>(0.0f);
        return;
    }
    const bool gated = d.act == GEMM_MOE_SWIGLU;
    const int per = gated ? 8 : 16;  // values of h per unit
    // (the host keeps units times steps below 2^30, and E and I keep units below 2^26)
    const int UB = static_cast<int>((d.I + per - 1) / per);
    if constexpr (NTMAX > 2) {
        // equal shares of the costs: a share's bounds are units, found in the expert that holds them
        const Share ctas(s.all_cost * UB, G);
        const int bound[2] = {ctas.lo(cta), ctas.lo(cta + 1)};
        for (int i = threadIdx.x; i < A; i += MT) {
            const int w = unit_cost(__popcll(s.mask[s.active[i]]));
            const int first = s.cost[i] * UB, next = first + w * UB;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (bound[k] >= first && (bound[k] < next || i == A - 1))
                    (k == 0 ? s.u_lo : s.u_hi) = i * UB + (bound[k] - first + w - 1) / w;
        }
    } else if (threadIdx.x == 0) {  // (one cost)
        const Share ctas(UB * A, G);
        s.u_lo = ctas.lo(cta);
        s.u_hi = ctas.lo(cta + 1);
    }
    __syncthreads();

    // ---------------------------------------------------------------- up
    const uint16_t* xp = reinterpret_cast<const uint16_t*>(a.ws + a.w.x);
    T* h = reinterpret_cast<T*>(a.ws + a.w.h);
    const int g = lane >> 2, t4 = lane & 3;
    float* my_tile = tiles + warp * 2 * TILE;
    {
        const int KS = static_cast<int>(a.w.hp / 64);
        const int u_lo = s.u_lo, n_u = s.u_hi - u_lo;
        // Whole units go to the warps in turn: all warps walk H together and find the tokens'
        // values in L1 (each x row comes from L2 once per 16 units).  The units left over are cut.
        const int whole = n_u / kMoeWarps, u_cut = u_lo + whole * kMoeWarps;
        const Share warps(n_u % kMoeWarps * KS, kMoeWarps);
        const int lo = warps.lo(warp), hi = warps.lo(warp + 1);
        const uint16_t* w1 = static_cast<const uint16_t*>(a.w1);
        const auto finish = [&](int u, const float (&acc)[NTMAX][4]) {
            const int e = s.active[u / UB];
            const int i0 = u % UB * per;
            const int n = __popcll(s.mask[e]), off = s.off[e];
            float top = 0.0f;  // the largest magnitude
#pragma unroll
            for (int j = 0; j < NTMAX; ++j) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = j * 8 + t4 * 2 + c;
                    if (col >= n) continue;
                    T* row = h + (off + col) * 2 * a.w.ip;
                    const float v0 = acc[j][c], v1 = acc[j][2 + c];
                    const auto put = [&](int i, float v) {
                        two_parts(row + i, a.w.ip, v);
                        top = fmaxf(top, fabsf(v));
                    };
                    if (gated) {
                        if (i0 + g < d.I) put(i0 + g, swiglu(v0, v1));
                    } else {
                        if (i0 + g < d.I) put(i0 + g, moe_act(d.act, v0));
                        if (i0 + g + 8 < d.I) put(i0 + g + 8, moe_act(d.act, v1));
                    }
                }
            }
            if constexpr (kMoeBig<T>) {
                if (top >= kMoeBigFrom) {
                    float copy[NTMAX][4];
#pragma unroll
                    for (int j = 0; j < NTMAX * 4; ++j) copy[j / 4][j % 4] = acc[j / 4][j % 4];
                    put_big<T, NTMAX>(a, copy, e, i0);
                }
            }
        };
        // Position in the warp's stream of steps -> unit, step.
        const auto at = [&](int pos, int& u, int& s0) {
            if (pos < whole * KS) {
                u = u_lo + pos / KS * kMoeWarps + warp;
                s0 = pos % KS;
            } else {
                const int q = pos - whole * KS + lo;
                u = u_cut + q / KS;
                s0 = q % KS;
            }
        };
        // Row r of a unit (rows past the last read it again: their sums are not used).
        const auto row = [&](int u, int r) {
            const int64_t i = u % UB * per + (gated ? r & 7 : r);
            return w1 + s.active[u / UB] * d.stride_w1 +
                   (min(i, d.I - 1) + (gated && r >= 8 ? d.I : 0)) * d.ld_w1;
        };
        const int total = whole * KS + hi - lo;
        int u = 0, s0 = 0, s1 = 0;
        for (int pos = 0; pos < total; pos += s1 - s0) {
            float acc[NTMAX][4] = {};
            at(pos, u, s0);
            s1 = min(KS, s0 + total - pos);
            const int e = s.active[u / UB];
            const int n = __popcll(s.mask[e]), off = s.off[e];
            with_groups<NTMAX>(n, [&](auto tag) {
                constexpr int NT = decltype(tag)::value;
                Columns<NT> x;
                x.base = xp;
#pragma unroll
                for (int j = 0; j < NT; ++j)  // columns past the last read its row: their sums are not used
                    x.set(j, s.slot_token[off + min(j * 8 + g, n - 1)] * static_cast<uint32_t>(KS));
                steps<T, ROWS, NT, NTMAX, 1>(row(u, g), row(u, g + 8), x, s0, s1, static_cast<int>(d.H), KS, t4, acc);
            });
            if (s0 == 0 && s1 == KS) {
                finish(u, acc);
            } else {
                // a unit that began in an earlier warp goes to this warp's first tile, one that
                // goes on in a later one to its second
                float* tile = my_tile + (s0 > 0 ? 0 : TILE);
#pragma unroll
                for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) tile[(j * 4 + c) * 32 + lane] = acc[j][c];
            }
        }
        __syncthreads();
        if (total > 0 && s0 == 0 && s1 < KS) {
            // this warp's last unit goes on in later ones: their sums, in order
            float acc[NTMAX][4];
#pragma unroll
            for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[j][c] = my_tile[TILE + (j * 4 + c) * 32 + lane];
            for (int w = warp + 1; w < kMoeWarps; ++w) {
                if (warps.lo(w) >= (u - u_cut + 1) * KS || warps.lo(w) == warps.lo(w + 1)) break;
                const float* tile = tiles + w * 2 * TILE;
#pragma unroll
                for (int j = 0; j < NTMAX; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[j][c] += tile[(j * 4 + c) * 32 + lane];
            }
            finish(u, acc);
        }
    }

    // ---------------------------------------------------------------- grid barrier
    // Four warps side by side take 16 of a block's columns each and walk the same steps
    // (sharing h in L1); four such teams share the CTA's steps.  The weights do not depend on
    // h: the first of them are asked into L2 before the barrier.
    const int sub = warp & 3, team = warp >> 2;
    const int OB = static_cast<int>((d.H + kMoeBlock - 1) / kMoeBlock);
    const int KS = static_cast<int>(a.w.ip / 64);
    const int block = A * KS;  // steps of an output block
    const Share ctas(OB * block, G);
    const int c_lo = ctas.lo(cta), c_hi = ctas.lo(cta + 1);
    const Share teams(c_hi - c_lo, kMoeTeams);
    const int lo = c_lo + teams.lo(team), hi = c_lo + teams.lo(team + 1);
    const uint16_t* w2 = static_cast<const uint16_t*>(a.w2);
    const auto row = [&](int v, int r) {
        const int64_t o = v / A * kMoeBlock + sub * 16 + r;
        return w2 + s.active[v % A] * d.stride_w2 + min(o, d.H - 1) * d.ld_w2;
    };
    if (lo < hi) {
        const int k = (lo % KS + t4) * 64;  // four steps of the warp's rows
        if (k < d.I) {
            prefetch_l2(row(lo / KS, g) + k);
            prefetch_l2(row(lo / KS, g + 8) + k);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned* bar = reinterpret_cast<unsigned*>(a.ws + a.w.bar);
        if (!((d.flags & GEMM_FLAG_TEST_STALL) && cta == 0))
            // (the low 16 bits count the CTAs, the high ones those that wrote a value beyond FP16)
            asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(bar), "r"(1u + (static_cast<unsigned>(s.big) << 16))
                         : "memory");
        const uint64_t t0 = globaltimer_ns();
        unsigned all;
        while (((all = ld_acquire_gpu(bar)) & 0xFFFFu) < static_cast<unsigned>(G)) {
            if (globaltimer_ns() - t0 > a.timeout_ns) {
                atomicOr(a.status, DEVERR_TIMEOUT);
                s.gave_up = 1;
                break;
            }
        }
        s.big = static_cast<int>(all >> 16);
    }
    __syncthreads();
    if (s.gave_up) return;

    // ---------------------------------------------------------------- down
    const int ytile = 16 * tok;  // [row][token] of a warp
    float* yt = my_tile;
    float* flushed = reinterpret_cast<float*>(a.ws + a.w.flushed) + ((cta * kMoeTeams + team) * kMoeBlock + sub * 16) * tok;
    for (int i = lane; i < ytile; i += 32) yt[i] = 0.0f;
    __syncwarp();
    const int first_ob = lo / block;
    if (sub == 0 && lane == 0) {
        s.team_first[team] = first_ob;
        s.team_last[team] = lo < hi ? (hi - 1) / block : -1;
    }
    for (int cur = lo, ob_now = first_ob; cur < hi;) {
        const int v = cur / KS;
        const int s0 = cur % KS, s1 = min(KS, s0 + hi - cur);
        const int ob = v / A;
        const int e = s.active[v - ob * A];
        const int n = __popcll(s.mask[e]), off = s.off[e];
        if (ob != ob_now) {
            // a team enters a second block at most: its sums of the first go to the workspace
            for (int i = lane; i < ytile; i += 32) {
                flushed[i] = yt[i];
                yt[i] = 0.0f;
            }
            ob_now = ob;
            __syncwarp();
        }
        float acc[NTMAX][4] = {};
        with_groups<NTMAX>(n, [&](auto tag) {
            constexpr int NT = decltype(tag)::value;
            Columns<NT> x;
            x.base = reinterpret_cast<const uint16_t*>(h);
#pragma unroll
            for (int j = 0; j < NT; ++j) x.set(j, static_cast<uint32_t>(off + min(j * 8 + g, n - 1)) * 2 * KS);
            steps<T, ROWS, NT, NTMAX, 2>(row(v, g), row(v, g + 8), x, s0, s1, static_cast<int>(d.I), KS, t4, acc);
        });
#pragma unroll
        for (int j = 0; j < NTMAX; ++j) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = j * 8 + t4 * 2 + c;
                if (col >= n) continue;
                const int t = s.slot_token[off + col];
                const float wgt = s.slot_weight[off + col];
                yt[g * tok + t] += wgt * acc[j][c];
                yt[(g + 8) * tok + t] += wgt * acc[j][2 + c];
            }
        }
        __syncwarp();
        cur += s1 - s0;
    }
    if constexpr (kMoeBig<T>) {
        if (s.big) add_big<T, NTMAX>(a);
    }
    __syncthreads();

    // Output blocks of this CTA: the sums of its warps, in order.
    T* y = static_cast<T*>(a.y);
    float* partial = reinterpret_cast<float*>(a.ws + a.w.partial);
    if (c_lo >= c_hi) return;
    const int ob_lo = c_lo / block, ob_hi = (c_hi - 1) / block;
    const int ysize = kMoeBlock * tok;
    const float* all_flushed = reinterpret_cast<const float*>(a.ws + a.w.flushed) + cta * kMoeTeams * ysize;
    for (int i = threadIdx.x; i < (ob_hi - ob_lo + 1) * ysize; i += MT) {
        const int ob = ob_lo + i / ysize, el = i % ysize;
        const int el_sub = el / ytile, el_in = el - el_sub * ytile;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kMoeTeams; ++w)
            if (ob == s.team_last[w])
                sum += tiles[(w * 4 + el_sub) * 2 * TILE + el_in];
            else if (ob == s.team_first[w] && ob < s.team_last[w])
                sum += all_flushed[w * ysize + el];
        if (ob * block >= c_lo && (ob + 1) * block <= c_hi) {
            const int o = ob * kMoeBlock + el / tok;
            if (o < d.H) y[(el % tok) * d.ldy + o] = cast16<T>(sum);
        } else {
            partial[(cta * 2 + (ob == ob_lo ? 0 : 1)) * ysize + el] = sum;
        }
    }
    // The first and the last block: whoever arrives last at a cut one joins it.
    if (ob_lo * block >= c_lo && (ob_hi + 1) * block <= c_hi) return;  // neither is cut
    __syncthreads();
    if (threadIdx.x < 2) {
        const int ob = threadIdx.x == 0 ? ob_lo : ob_hi;
        const bool whole = ob * block >= c_lo && (ob + 1) * block <= c_hi;
        int last = 0;
        if (!whole && (threadIdx.x == 0 || ob_hi != ob_lo)) {
            // blocks are cut between neighbours, none of which is empty
            const unsigned parts = ctas.owner((ob + 1) * block - 1) - ctas.owner(ob * block) + 1;
            unsigned* ctr = reinterpret_cast<unsigned*>(a.ws + a.w.counters);
            // releases the CTA's partial sums (written before the barrier), acquires the others'
            unsigned before;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(ctr + ob) : "memory");
            last = before == parts - 1;
        }
        s.last[threadIdx.x] = last;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!s.last[k]) continue;
        const int ob = k == 0 ? ob_lo : ob_hi;
        const int from = ctas.owner(ob * block), to = ctas.owner((ob + 1) * block - 1);
        // (the first of them may have begun in an earlier block: then this one is its last)
        const int first = from * 2 + (ctas.lo(from) >= ob * block ? 0 : 1);
        for (int i = threadIdx.x; i < ysize / 4; i += MT) {
            const auto part = [&](int slot) {
                return __ldcg(reinterpret_cast<const float4*>(partial + static_cast<int64_t>(slot) * ysize) + i);
            };
            float4 sum = part(first);
            for (int c = from + 1; c <= to; c += 8) {  // eight reads in flight, added in order
                float4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = part(min(c + j, to) * 2);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j <= to) {
                        sum.x += v[j].x;
                        sum.y += v[j].y;
                        sum.z += v[j].z;
                        sum.w += v[j].w;
                    }
            }
            const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int el = 4 * i + j, o = ob * kMoeBlock + el / tok;
                if (o < d.H) y[(el % tok) * d.ldy + o] = cast16<T>(out[j]);
            }
        }
    }
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

template <typename T, int ROWS, int NTMAX, bool GIVEN>
cudaError_t launch_experts(const MoeArgs& a, int grid, cudaStream_t st) {
    auto k = moe_experts_kernel<T, ROWS, NTMAX, GIVEN>;
    constexpr int smem = kMoeSmem<NTMAX>;
    static_assert(smem <= 232448, "shared memory");
    static std::atomic<unsigned char> ready[kMaxDevices];
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (ce != cudaSuccess) return ce;
        if (dev < kMaxDevices) ready[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(MT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;  // the grid barrier needs every CTA resident
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T, int ROWS, bool GIVEN>
cudaError_t launch_t(const MoeArgs& a, int grid, cudaStream_t st) {
    const unsigned blocks = GIVEN
                                ? static_cast<unsigned>(std::min<int64_t>((a.d.T * a.w.hp / 8 + RT - 1) / RT, grid))
                                : static_cast<unsigned>((a.d.E + RE - 1) / RE * ((a.d.T + RTOK - 1) / RTOK));
    // the router's rows and x take vector loads on their own terms
    const bool rvec = (GIVEN || (reinterpret_cast<uintptr_t>(a.router) % 16 == 0 && a.d.ld_router % 8 == 0)) &&
                      reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.d.ldx % 8 == 0 && a.d.H % 8 == 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(RT);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (it waits before its first read)
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t ce = cudaLaunchKernelEx(&cfg, rvec ? moe_router_kernel<T, true, GIVEN> : moe_router_kernel<T, false, GIVEN>, a);
    if (ce != cudaSuccess) return ce;
    // groups of 8 tokens that one expert can be given: 1, 2, 4 or 8
    if (a.d.T <= 8) return launch_experts<T, ROWS, 1, GIVEN>(a, grid, st);
    if (a.d.T <= 16) return launch_experts<T, ROWS, 2, GIVEN>(a, grid, st);
    if (a.d.T <= 32) return launch_experts<T, ROWS, 4, GIVEN>(a, grid, st);
    return launch_experts<T, ROWS, 8, GIVEN>(a, grid, st);
}

template <bool GIVEN>
cudaError_t launch_moe_kernels(const MoeArgs& a, int grid, cudaStream_t st) {
    const auto all = [&](int64_t n) {  // every row on n elements, rows a multiple of n long
        return reinterpret_cast<uintptr_t>(a.w1) % (2 * n) == 0 && reinterpret_cast<uintptr_t>(a.w2) % (2 * n) == 0 &&
               a.d.ld_w1 % n == 0 && a.d.ld_w2 % n == 0 && a.d.stride_w1 % n == 0 && a.d.stride_w2 % n == 0 &&
               a.d.H % n == 0 && a.d.I % n == 0;
    };
    const bool f16 = a.d.dtype == GEMM_F16;
    if (all(16)) return f16 ? launch_t<__half, ROWS_32, GIVEN>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_32, GIVEN>(a, grid, st);
    if (all(8)) return f16 ? launch_t<__half, ROWS_16, GIVEN>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_16, GIVEN>(a, grid, st);
    return f16 ? launch_t<__half, ROWS_ANY, GIVEN>(a, grid, st) : launch_t<__nv_bfloat16, ROWS_ANY, GIVEN>(a, grid, st);
}

}  // namespace
}  // namespace g13
