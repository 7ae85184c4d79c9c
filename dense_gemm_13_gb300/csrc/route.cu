// route.cu -- the experts of each token, from its logits z:
//
//   s = softmax(z) or sigmoid(z);   c = s + bias, or without a bias z itself (the same order)
//   with groups: of each group of E / groups experts the best c, or the sum of the two best s + bias; the
//   top_groups best groups stay
//   the top_k experts with the largest c among them (equal ones: the lowest index), and of each
//   s * scale, or s * scale / (the sum of their s)
//
// A token is a warp's: each lane holds every 32nd logit, and a round finds the largest key by one
// warp-wide reduction and the lowest index that has it by another.  Warps take tokens in turn, persistent.
//
// The order has to be that of the exact c.  Logits are compared as they are; where c is a sum, it is computed in FP32
// and is off by at most `delta`.  Two neighbours in the chosen order (or two groups at the border) that
// are not further apart than the errors allow send the token through the same steps in 64 bits, which a token in
// some thousands needs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "route.h"

namespace g13 {
namespace {

constexpr int RW = 8;  // warps of a CTA, a token each
constexpr unsigned ALL = 0xFFFFFFFFu;

// Order-preserving keys: 0 is "not there", 1 a NaN, -0 and +0 the same.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key <= 1u) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (v != v) return 1ull;
    const unsigned long long b = __double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 1ull << 63);
}
__device__ __forceinline__ double value_of(unsigned long long key) {
    if (key <= 1ull) return __longlong_as_double(0x7FFFFFFFFFFFFFFFll);
    return __longlong_as_double(key >> 63 ? key & 0x7FFFFFFFFFFFFFFFull : ~key);
}

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
    const int64_t i = t * a.d.ld + e;
    if (a.d.dtype == GEMM_F32) return __ldg(static_cast<const float*>(a.logits) + i);
    if (a.d.dtype == GEMM_BF16) return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(a.logits) + i));
    return __half2float(__ldg(static_cast<const __half*>(a.logits) + i));
}

// The two best keys of `lanes` neighbouring lanes.
template <typename K>
__device__ __forceinline__ void best_two(K& b1, K& b2, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) {
        const K o1 = __shfl_xor_sync(ALL, b1, o), o2 = __shfl_xor_sync(ALL, b2, o);
        b2 = max(min(b1, o1), max(b2, o2));
        b1 = max(b1, o1);
    }
}

// The group that a lane stands for: `lanes` neighbours scan one group.
struct Groups {
    int lanes, mine, sub, per;
    __device__ __forceinline__ Groups(const gemm_route_desc_t& d, int lane) {
        int n = 1;
        while (n < d.groups) n *= 2;
        lanes = 32 / n;
        mine = lane / lanes;
        sub = lane % lanes;
        per = static_cast<int>(d.E / d.groups);
    }
};
// Bits (at each group's first lane) of the top_groups largest keys; equal ones: the lowest index.
template <typename K>
__device__ __forceinline__ unsigned keep_groups(const gemm_route_desc_t& d, const Groups& g, K key) {
    int before = 0;
    for (int j = 0; j < static_cast<int>(d.groups); ++j) {
        const K o = __shfl_sync(ALL, key, j * g.lanes);
        before += o > key || (o == key && j < g.mine);
    }
    return __ballot_sync(ALL, g.sub == 0 && g.mine < d.groups && before < d.top_groups);
}

// A token in 64 bits, c of its experts in `c` (shared, this warp's).  Lane j < top_k gets expert j.
__device__ __noinline__ int choose64(const RouteArgs& a, int64_t t, double* c, int lane) {
    const gemm_route_desc_t& d = a.d;
    const int E = static_cast<int>(d.E);
    const bool softmax = d.scores == GEMM_ROUTE_SOFTMAX;
    double top = -INFINITY, sum = 0.0;
    if (softmax) {
        for (int e = lane; e < E; e += 32) top = fmax(top, static_cast<double>(logit(a, t, e)));
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(ALL, top, o));
        for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(logit(a, t, e)) - top);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    const auto score = [&](int e) {
        const double z = static_cast<double>(logit(a, t, e));
        return (softmax ? exp(z - top) / sum : 1.0 / (1.0 + exp(-z))) +
               (a.bias ? static_cast<double>(__ldg(a.bias + e)) : 0.0);
    };
    const bool by_score = a.bias != nullptr;  // what experts are compared by (else the logits)
    const bool sums = d.groups > d.top_groups && d.group_score == GEMM_ROUTE_GROUP_TOP2;
    __syncwarp();
    for (int e = lane; e < E; e += 32) c[e] = by_score || sums ? score(e) : static_cast<double>(logit(a, t, e));
    __syncwarp();
    const Groups g(d, lane);
    unsigned kept = ALL;
    if (d.groups > d.top_groups) {
        unsigned long long b1 = 0, b2 = 0;
        if (g.mine < d.groups)
            for (int i = g.sub; i < g.per; i += g.lanes) {
                const unsigned long long k = key_of(c[g.mine * g.per + i]);
                b2 = max(min(b1, k), b2);
                b1 = max(b1, k);
            }
        best_two(b1, b2, g.lanes);
        if (sums && g.per > 1) b1 = key_of(value_of(b1) + value_of(b2));
        kept = keep_groups(d, g, g.mine < d.groups ? b1 : 0ull);
    }
    __syncwarp();
    if (!by_score && sums)
        for (int e = lane; e < E; e += 32) c[e] = static_cast<double>(logit(a, t, e));
    __syncwarp();
    int mine = 0;
    unsigned taken = 0;  // of this lane's experts (at most 16)
    for (int j = 0; j < static_cast<int>(d.top_k); ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
        for (int i = 0, e = lane; e < E; ++i, e += 32) {
            if ((taken >> i & 1u) || !(kept >> (d.groups > d.top_groups ? e / g.per * g.lanes : 0) & 1u)) continue;
            const unsigned long long k = key_of(c[e]);
            if (k > best) best = k, at = e;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long ob = __shfl_xor_sync(ALL, best, o);
            const int oa = __shfl_xor_sync(ALL, at, o);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
        if (at % 32 == lane) taken |= 1u << (at / 32);
        if (j == lane) mine = at;
    }
    return mine;
}

// PER: logits of a lane.
template <int PER>
__global__ void __launch_bounds__(RW * 32) route_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(8) double shared[RW][PER * 32];
    const gemm_route_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = static_cast<int>(d.E), top_k = static_cast<int>(d.top_k);
    float* mine = reinterpret_cast<float*>(shared[warp]);
    const bool softmax = d.scores == GEMM_ROUTE_SOFTMAX, grouped = d.groups > d.top_groups;
    const bool by_score = a.bias != nullptr;
    const bool sums = grouped && d.group_score == GEMM_ROUTE_GROUP_TOP2;
    const Groups g(d, lane);
    float bias[PER];
    int group_bit[PER];  // the ballot's bit of each expert's group
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        bias[i] = by_score && e < E ? __ldg(a.bias + e) : 0.0f;
        group_bit[i] = grouped && e < E ? e / g.per * g.lanes : 0;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * RW + warp; t < d.T; t += static_cast<int64_t>(gridDim.x) * RW) {
        float z[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) z[i] = i * 32 + lane < E ? logit(a, t, i * 32 + lane) : -INFINITY;
        // scores
        float top = 0.0f, sum = 1.0f;
        if (softmax) {
            top = z[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
            sum = 0.0f;
        }
        float c[PER];  // s + bias
        if (softmax) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[i] = i * 32 + lane < E ? expf(z[i] - top) : 0.0f;
                sum += c[i];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = fmaf(c[i], inv, bias[i]);
        } else if (by_score || sums) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = 1.0f / (1.0f + expf(-z[i])) + bias[i];
        }
        // How far c may be off, apart from its own rounding (2^-23 |c|): a sigmoid s by 2^-22 (its slope against
        // z's relative steps, s (1 - s) |z|, stays below 0.23); a softmax by 2^-17 of itself, up to
        // exponents of -60, below which s is nothing, so by 2^-17 of the largest.
        const float delta = softmax ? 0x1p-17f / sum : 0x1p-21f;
        bool unsure = false;
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = i * 32 + lane < E ? key_of(by_score ? c[i] : z[i]) : 0u;
        if (grouped) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i * 32 + lane < E) mine[i * 32 + lane] = by_score || sums ? c[i] : z[i];
            __syncwarp();
            uint32_t b1 = 0, b2 = 0;
            if (g.mine < d.groups)
                for (int i = g.sub; i < g.per; i += g.lanes) {
                    const uint32_t k = key_of(mine[g.mine * g.per + i]);
                    b2 = max(min(b1, k), b2);
                    b1 = max(b1, k);
                }
            best_two(b1, b2, g.lanes);
            if (sums && g.per > 1) b1 = key_of(value_of(b1) + value_of(b2));
            if (g.mine >= d.groups) b1 = 0u;
            const unsigned kept = keep_groups(d, g, b1);
            if (by_score || sums) {
                // the worst group that stays and the best that goes
                const bool stays = kept >> (g.mine * g.lanes) & 1u;
                const float lo = value_of(__reduce_min_sync(ALL, stays ? b1 : ALL));
                const float hi = value_of(__reduce_max_sync(ALL, stays ? 0u : b1));
                unsure = !(lo - hi > 4.0f * delta + 0x1p-20f * (fabsf(lo) + fabsf(hi)));
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!(kept >> group_bit[i] & 1u)) key[i] = 0u;
        }
        // the choice: lane j keeps expert j
        int id = 0;
        float before = INFINITY;
        for (int j = 0; j <= top_k; ++j) {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) m = max(m, key[i]);
            m = __reduce_max_sync(ALL, m);
            if (by_score && m != 0u) {
                const float v = value_of(m);
                if (j > 0) unsure = unsure || !(before - v > 2.0f * delta + 0x1p-21f * (fabsf(before) + fabsf(v)));
                before = v;
            }
            if (j == top_k) break;
            uint32_t e = 0xFFFFu;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == m) e = i * 32 + lane;
            e = __reduce_min_sync(ALL, e);
            if (lane == j) id = static_cast<int>(e);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i * 32 + lane == e) key[i] = 0u;
        }
        if (unsure) id = choose64(a, t, shared[warp], lane);
        // the weights
        float w = 0.0f;
        if (lane < top_k) {
            const float v = logit(a, t, id);
            w = softmax ? expf(v - top) / sum : 1.0f / (1.0f + expf(-v));
        }
        if (d.normalize) {
            float all = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(ALL, all, o);
            w /= all;
        }
        if (lane < top_k) {
            a.ids[t * top_k + lane] = id;
            a.weights[t * top_k + lane] = w * d.scale;
        }
    }
}

template <int PER>
cudaError_t launch(const RouteArgs& a, int num_sms, cudaStream_t st) {
    const int64_t blocks = (a.d.T + RW - 1) / RW;
    route_kernel<PER><<<static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(num_sms) * 6)), RW * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t st) {
    const int64_t E = a.d.E;
    if (E <= 32) return launch<1>(a, num_sms, st);
    if (E <= 64) return launch<2>(a, num_sms, st);
    if (E <= 128) return launch<4>(a, num_sms, st);
    if (E <= 256) return launch<8>(a, num_sms, st);
    return launch<16>(a, num_sms, st);
}

}  // namespace g13
