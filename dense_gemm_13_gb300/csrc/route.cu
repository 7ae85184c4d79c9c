// route.cu -- the experts of each token, from its logits z:
//
//   s = softmax(z) or sigmoid(z);   c = s + bias, or without a bias z itself (the same order)
//   with groups: of each group of E / groups experts the best c, or the sum of the two best s + bias; the
//   top_groups best groups stay
//   the top_k experts with the largest c among them (equal ones: the lowest index), and of each
//   s * scale, or s * scale / (the sum of their s)
//
// A token is a warp's: each lane holds every 32nd logit, as an integer that orders like the number, with its place in
// the lane in the lowest bits, and sorts its own.  A round of the choice is one warp-wide maximum of the lanes' best and a
// vote on who has it; that lane moves its others up.  Warps take tokens in turn, persistent.  Up to a few hundred
// tokens the launch is the cost; with many the instructions are.
//
// The order has to be that of the exact c.  16-bit logits leave the lowest bits free.  FP32 logits lose up to four bits
// to the place, and where c is a sum it is computed in FP32 and off by `delta`.  Where these leave two neighbours in
// the chosen order, or groups at the border, in doubt, the experts that can be meant are worked out in 64 bits, one a
// lane, and ranked; with more than 32 of them, or a NaN, the token goes through all steps in 64 bits.  Of random tokens
// that is one in a thousand.  (An FP64 operation of a warp takes some 64 cycles here: 1.5 us for a score, 18 us for all
// 256 of a token, as long as 16384 tokens without doubt take together.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "route.h"

namespace g13 {
namespace {

constexpr int RW = 8;  // warps of a CTA, a token each
constexpr unsigned ALL = 0xFFFFFFFFu;

// An integer that orders like the number (-0 below +0; add 0 first), and back.
constexpr int NONE = -0x7FFFFFFF - 1;  // not there
__device__ __forceinline__ int ordered(float v) {
    const int b = __float_as_int(v);
    return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float number(int k) { return __int_as_float(k ^ (k >> 31 & 0x7FFFFFFF)); }
// In 64 bits 0 is "not there" and 1 a NaN, -0 and +0 are the same.
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (v != v) return 1ull;
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
    return (b >> 63) ? ~b : (b | 1ull << 63);
}
__device__ __forceinline__ double value_of(unsigned long long key) {
    if (key <= 1ull) return __longlong_as_double(0x7FFFFFFFFFFFFFFFll);
    return __longlong_as_double(key >> 63 ? key & 0x7FFFFFFFFFFFFFFFull : ~key);
}

// PER logits of a lane, every 32nd; those past the last are -infinity (FULL: there are none).
template <int PER, bool FULL>
__device__ __forceinline__ void logits(const RouteArgs& a, int64_t t, int lane, float (&z)[PER]) {
    const int E = static_cast<int>(a.d.E);
    const int64_t at = t * a.d.ld + lane;
    if (a.d.dtype == GEMM_F32) {
        const float* p = static_cast<const float*>(a.logits) + at;
#pragma unroll
        for (int i = 0; i < PER; ++i) z[i] = FULL || i * 32 + lane < E ? __ldg(p + i * 32) : -INFINITY;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.logits) + at;
        uint16_t v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = FULL || i * 32 + lane < E ? __ldg(p + i * 32) : uint16_t(0);
        if (a.d.dtype == GEMM_BF16) {
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] = __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] = __half2float(__ushort_as_half(v[i]));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (!FULL && i * 32 + lane >= E) z[i] = -INFINITY;
    }
}
// Falls from the first to the last: Batcher's odd-even merge sort (1968).
template <int PER>
__device__ __forceinline__ void sort_down(int (&k)[PER]) {
#pragma unroll
    for (int p = 1; p < PER; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < PER; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < PER && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const int hi = max(k[i + j], k[i + j + q]), lo = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                        k[i + j + q] = lo;
                    }
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
__device__ __forceinline__ unsigned keep_groups(const gemm_route_desc_t& d, const Groups& g, unsigned long long key) {
    int before = 0;
    for (int j = 0; j < static_cast<int>(d.groups); ++j) {
        const unsigned long long o = __shfl_sync(ALL, key, j * g.lanes);
        before += o > key || (o == key && j < g.mine);
    }
    return __ballot_sync(ALL, g.sub == 0 && g.mine < d.groups && before < d.top_groups);
}

// e^x of four numbers in 64 bits: x = n ln 2 + r, 2^n times Taylor's series of e^r to r^13 (|r| <= 0.35: the next term is
// below 2^-57).  Arguments beyond +-700 count as these.
template <int N>
struct Doubles {
    double v[N];
};
template <int N>
__device__ __noinline__ Doubles<N> exp64(Doubles<N> x) {
    constexpr double LOG2E = 1.4426950408889634074;
    constexpr double LN2_HI = 0.693147180559890330, LN2_LO = 5.497923018708371e-14;  // ln 2: 42 bits, and the rest
    double n[N], r[N], p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const double c = x.v[i] > 700.0 ? 700.0 : x.v[i] < -700.0 ? -700.0 : x.v[i];
        n[i] = rint(c * LOG2E);
        r[i] = fma(-n[i], LN2_LO, fma(-n[i], LN2_HI, c));
        p[i] = 1.0 / 6227020800.0;  // 1 / 13!
    }
    const double inv[13] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                            1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
#pragma unroll
    for (int k = 12; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = fma(p[i], r[i], inv[k]);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (x.v[i] == x.v[i])
            x.v[i] = __longlong_as_double(__double_as_longlong(p[i]) + (static_cast<long long>(static_cast<int>(n[i])) << 52));
    return x;
}
// c of a token's experts in 64 bits.
struct Score64 {
    const RouteArgs& a;
    int64_t t;
    double top = 0.0, sum = 1.0;
    __device__ __forceinline__ double arg(int e) const {
        const double z = e < a.d.E ? static_cast<double>(logit(a, t, e)) : 0.0;
        return a.d.scores == GEMM_ROUTE_SOFTMAX ? z - top : -z;
    }
    // e^arg of experts e, e + 32, e + 64, e + 96
    __device__ __forceinline__ Doubles<4> four(int e) const {
        return exp64(Doubles<4>{arg(e), arg(e + 32), arg(e + 64), arg(e + 96)});
    }
    __device__ Score64(const RouteArgs& args, int64_t token, int lane) : a(args), t(token) {
        if (a.d.scores != GEMM_ROUTE_SOFTMAX) return;
        const int E = static_cast<int>(a.d.E);
        float m = -INFINITY;
        for (int e = lane; e < E; e += 32) m = fmaxf(m, logit(a, t, e));
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(ALL, m, o));
        top = static_cast<double>(m);
        sum = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 128) {
            const Doubles<4> x = four(e);
            sum += (x.v[0] + (e + 32 < E ? x.v[1] : 0.0)) + ((e + 64 < E ? x.v[2] : 0.0) + (e + 96 < E ? x.v[3] : 0.0));
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    // c from e^arg
    __device__ __forceinline__ double of(int e, double x) const {
        const bool softmax = a.d.scores == GEMM_ROUTE_SOFTMAX;
        return (softmax ? x : 1.0) / (softmax ? sum : 1.0 + x) + (a.bias ? static_cast<double>(__ldg(a.bias + e)) : 0.0);
    }
};

// The experts `id` of the first n lanes (at most 32) in the order of their c (without a bias: of their logits); lane j
// gets the one that comes j-th.  room: 32 numbers of this warp's shared memory.
__device__ __noinline__ int rank64(const RouteArgs& a, int64_t t, int id, int n, int* room, int lane) {
    unsigned long long key = 0;
    if (a.bias) {
        const Score64 score(a, t, lane);
        const Doubles<1> x = exp64(Doubles<1>{lane < n ? score.arg(id) : 0.0});
        if (lane < n) key = key_of(score.of(id, x.v[0]));
    } else if (lane < n) {
        key = key_of(static_cast<double>(logit(a, t, id)));
    }
    int before = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const unsigned long long o = __shfl_sync(ALL, key, j);
        const int oid = __shfl_sync(ALL, id, j);
        before += o > key || (o == key && oid < id);
    }
    __syncwarp();
    if (lane < n) room[before] = id;
    __syncwarp();
    return lane < n ? room[lane] : 0;
}

// Of the groups in `open` (bits at their first lanes) the `need` with the largest exact score, as such bits.  id: the
// experts that can count for them, one in each of the first n lanes.
__device__ __noinline__ unsigned keep64(const RouteArgs& a, int64_t t, int id, int n, unsigned open, int need, bool two, int lane) {
    const Score64 score(a, t, lane);
    const Doubles<1> x = exp64(Doubles<1>{lane < n ? score.arg(id) : 0.0});
    const unsigned long long key = lane < n ? key_of(score.of(id, x.v[0])) : 0ull;
    const Groups g(a.d, lane);
    const int at = lane < n ? id / g.per * g.lanes : -1;  // its group's first lane
    unsigned long long mine = 0;
    for (unsigned left = open; left != 0; left &= left - 1) {
        const int first = __ffs(left) - 1;
        unsigned long long b1 = at == first ? key : 0ull, b2 = 0;
        best_two(b1, b2, 32);
        if (two) b1 = key_of(value_of(b1) + value_of(b2));
        if (lane == first) mine = b1;
    }
    unsigned kept = 0;
    for (int j = 0; j < need; ++j) {
        unsigned long long best = mine, other = 0;
        best_two(best, other, 32);
        const int who = __ffs(__ballot_sync(ALL, mine == best && (open >> lane & 1u) && !(kept >> lane & 1u))) - 1;
        if (who < 0) break;
        kept |= 1u << who;
        if (lane == who) mine = 0;
    }
    return kept;
}

// A token in 64 bits, the keys of its experts in `key` (shared, this warp's).  Lane j < top_k gets expert j.
__device__ __noinline__ int choose64(const RouteArgs& a, int64_t t, unsigned long long* key, int lane) {
    const gemm_route_desc_t& d = a.d;
    const int E = static_cast<int>(d.E);
    const Score64 score(a, t, lane);
    const bool by_score = a.bias != nullptr;  // what experts are compared by (else the logits)
    const bool sums = d.groups > d.top_groups && d.group_score == GEMM_ROUTE_GROUP_TOP2;
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < E; e += 128) {
        const Doubles<4> x = score.four(e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = e + 32 * i;
            if (o < E) key[o] = key_of(by_score || sums ? score.of(o, x.v[i]) : static_cast<double>(logit(a, t, o)));
        }
    }
    __syncwarp();
    const Groups g(d, lane);
    unsigned kept = ALL;
    if (d.groups > d.top_groups) {
        unsigned long long b1 = 0, b2 = 0;
        if (g.mine < d.groups)
            for (int i = g.sub; i < g.per; i += g.lanes) {
                const unsigned long long k = key[g.mine * g.per + i];
                b2 = max(min(b1, k), b2);
                b1 = max(b1, k);
            }
        best_two(b1, b2, g.lanes);
        if (sums && g.per > 1) b1 = key_of(value_of(b1) + value_of(b2));
        kept = keep_groups(d, g, g.mine < d.groups ? b1 : 0ull);
    }
    __syncwarp();
    if (!by_score && sums)
        for (int e = lane; e < E; e += 32) key[e] = key_of(static_cast<double>(logit(a, t, e)));
    __syncwarp();
    for (int e = lane; e < E; e += 32)
        if (!(kept >> (d.groups > d.top_groups ? e / g.per * g.lanes : 0) & 1u)) key[e] = 0;
    int mine = 0;
    for (int j = 0; j < static_cast<int>(d.top_k); ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll 1
        for (int e = lane; e < E; e += 32)  // (the lane's own)
            if (key[e] > best) best = key[e], at = e;
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long ob = __shfl_xor_sync(ALL, best, o);
            const int oa = __shfl_xor_sync(ALL, at, o);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
        if (at % 32 == lane) key[at] = 0;
        if (j == lane) mine = at;
    }
    __syncwarp();
    return mine;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// PER: logits of a lane, a power of two.  FULL: E is 32 PER.
template <int PER, bool FULL>
__global__ void __launch_bounds__(RW * 32, PER == 16 ? 2 : 3) route_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ unsigned long long shared[RW][PER * 33];
    constexpr int PLACE = PER - 1;  // the bits of a key that hold the logit's place in its lane
    constexpr float LOG2E = 1.4426950408889634f;
    const gemm_route_desc_t& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = static_cast<int>(d.E), top_k = static_cast<int>(d.top_k);
    int* mine = reinterpret_cast<int*>(shared[warp]);  // whole keys: expert e at e + e / 32
    const bool softmax = d.scores == GEMM_ROUTE_SOFTMAX, grouped = d.groups > d.top_groups;
    const bool by_score = a.bias != nullptr;
    const bool sums = grouped && d.group_score == GEMM_ROUTE_GROUP_TOP2;
    const bool wide = d.dtype == GEMM_F32;
    const Groups g(d, lane);
    const bool has_group = g.mine < d.groups;
    float bias[PER];
    int group_bit[PER];  // the ballot's bit of each expert's group
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        bias[i] = by_score && e < E ? __ldg(a.bias + e) : 0.0f;
        group_bit[i] = grouped && e < E ? e / g.per * g.lanes : 0;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * RW + warp; t < d.T; t += static_cast<int64_t>(gridDim.x) * RW) {
        float z[PER], c[PER];  // c: s + bias
        logits<PER, FULL>(a, t, lane, z);
        float top = 0.0f, sum = 1.0f;
        if (softmax) {
            top = z[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
            top = number(__reduce_max_sync(ALL, ordered(top)));
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[i] = ex2((z[i] - top) * LOG2E);
                sum += FULL || i * 32 + lane < E ? c[i] : 0.0f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
            const float inv = rcp(sum);
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = fmaf(c[i], inv, bias[i]);
        } else if (by_score || sums) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = rcp(1.0f + ex2(z[i] * -LOG2E)) + bias[i];
        }
        // How far c may be off, apart from its own rounding (2^-24 |c|).  A sigmoid s by 1.1 * 2^-22: ex2 by 2^-22 of its value,
        // which counts s (1 - s) <= 1/4, its argument's roundings by 2^-24 and LOG2E's by 2^-26 of it, and s (1 - s) |z| <= 0.23;
        // 1 + e and rcp by 3 * 2^-24.  Of two softmax scores the difference by 2 * 2^-19 of the largest, 1 / sum, with 1 = 2^-23:
        // their common factor by 10 (a sum of 16 in a lane and five steps, half a unit each), 2 (ex2), 7 (the arguments' 1.12 |z - max|,
        // whose mean over the scores is at most ln E - ln sum <= 6.3) and 1 (rcp), 20 times a difference of at most
        // the largest; each by ex2 and its argument, (2 + 1.12 |z - max|) s, at most 2 of the largest: 24 <= 2 * 16.  Of two sums of two the same twice.
        const float delta = softmax ? 0x1p-19f * rcp(sum) : 0x1.2p-22f;
        bool unsure = softmax && sum != sum;
        int key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = ordered(by_score ? c[i] : z[i] + 0.0f);
        if (grouped || by_score) {
            __syncwarp();
            if (sums && !by_score) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (FULL || i * 32 + lane < E) mine[i * 33 + lane] = ordered(c[i]);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (FULL || i * 32 + lane < E) mine[i * 33 + lane] = key[i];
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = FULL || i * 32 + lane < E ? (key[i] & ~PLACE) | (PLACE - i) : NONE;
        if (grouped) {
            int b1 = NONE, b2 = NONE;
            if (has_group)
                for (int e = g.mine * g.per + g.sub, end = (g.mine + 1) * g.per; e < end; e += g.lanes) {
                    const int k = mine[e + (e >> 5)];
                    b2 = max(min(b1, k), b2);
                    b1 = max(b1, k);
                }
            best_two(b1, b2, g.lanes);
            float size = 0.0f;  // what the roundings of a sum's terms go by (biases of both signs may cancel)
            if (sums && g.per > 1) {
                const float c1 = number(b1), c2 = number(b2), both = c1 + c2 + 0.0f;
                if (has_group && fabsf(both) < INFINITY) size = fabsf(c1) + fabsf(c2);
                b1 = ordered(both);
            }
            if (!has_group || g.sub != 0) b1 = NONE;
            const int its_score = b1, second = sums && g.per > 1 ? b2 : b1;
            unsigned kept = 0;
            int lowest = 0, most = NONE;  // the worst group that stays and the best that goes
            for (int j = 0; j <= static_cast<int>(d.top_groups); ++j) {
                most = __reduce_max_sync(ALL, b1);
                if (j == 0) unsure = unsure || most > 0x7F800000;  // a NaN
                if (j == static_cast<int>(d.top_groups)) break;
                const int who = __ffs(__ballot_sync(ALL, b1 == most)) - 1;
                kept |= 1u << who;
                if (lane == who) b1 = NONE;
                lowest = most;
            }
            if (by_score || sums) {
                const float lo = number(lowest), hi = number(most);
                // (of each group: 2^-24 of its terms' sizes, and of their sum; an infinity is exact where it is not a sum)
                size = __int_as_float(__reduce_max_sync(ALL, __float_as_int(size)));
                const auto finite = [](float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; };
                const float off = 4.0f * delta + 0x1.8p-23f * (finite(lo) + finite(hi)) + 0x1.1p-23f * size;
                const bool sure = lo - hi > off || (!sums && lo == hi && !(fabsf(lo) < INFINITY));
                if (!unsure && !sure && !(fabsf(lo) < INFINITY)) {
                    unsure = true;
                } else if (!unsure && !sure) {
                    // the groups that may go either way, and of each the experts that may be its best (two)
                    const float v = number(its_score);
                    const unsigned open = __ballot_sync(ALL, its_score != NONE && v >= hi - off && v <= lo + off);
                    int n = 0, id = 0;
#pragma unroll 1
                    for (int i = 0; i < PER; ++i) {
                        const int e = i * 32 + lane, first = e < E ? e / g.per * g.lanes : 0;
                        const float least = number(__shfl_sync(ALL, second, first));
                        const bool may = e < E && (open >> first & 1u) &&
                                         number(mine[i * 33 + lane]) >= least - 2.0f * delta - 0x1p-22f * fabsf(least);
                        for (unsigned left = __ballot_sync(ALL, may); left != 0; left &= left - 1, ++n)
                            if (lane == n) id = i * 32 + __ffs(left) - 1;
                    }
                    kept &= ~open;
                    if (n <= 32)
                        kept |= keep64(a, t, id, n, open, static_cast<int>(d.top_groups) - __popc(kept), sums && g.per > 1, lane);
                    else
                        unsure = true;
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!(kept >> group_bit[i] & 1u)) key[i] = NONE;
        }
        // the choice: lane j keeps expert j (lane top_k the best of those that are left) and its key
        sort_down(key);
        int id = 0, its_key = NONE;
        for (int j = 0; j <= top_k; ++j) {
            const int best = __reduce_max_sync(ALL, key[0]);
            const int who = __ffs(__ballot_sync(ALL, key[0] == best)) - 1;
            if (lane == j) {
                id = (PLACE - (best & PLACE)) * 32 + who;
                its_key = best;
            }
            if (j == top_k) break;
            if (lane == who) {
#pragma unroll
                for (int i = 0; i + 1 < PER; ++i) key[i] = key[i + 1];
                key[PER - 1] = NONE;
            }
        }
        // a NaN, or nothing left that is needed: in 64 bits
        unsure = unsure || __any_sync(ALL, lane < top_k && (its_key > (0x7F800000 | PLACE) || its_key == NONE));
        // neighbours that are too close (of the ones left, another may be up to 2^-19 above the best by its key)
        if (by_score || wide) {
            const bool there = its_key != NONE;
            const int whole = by_score && there ? mine[id + (id >> 5)] : its_key;
            const int above = __shfl_up_sync(ALL, whole, 1);
            bool close = (above & ~PLACE) == (whole & ~PLACE);
            if (by_score) {
                const float u = number(above), v = number(whole);
                close = !(u - v > 2.0f * delta + (lane == top_k ? 0x1p-19f : 0x1p-23f) * (fabsf(u) + fabsf(v)));
            }
            bool doubt = __any_sync(ALL, close && there && lane > 0 && lane <= top_k);
            const int last = __shfl_sync(ALL, whole, top_k - 1);
            if (top_k == 32) {  // (no lane has looked at the next one)
                const int next = __reduce_max_sync(ALL, key[0]);
                const float u = number(last), v = number(next | PLACE);
                doubt = doubt || (next != NONE && (by_score ? !(u - v > 2.0f * delta + 0x1p-19f * (fabsf(u) + fabsf(v)))
                                                            : (next & ~PLACE) == (last & ~PLACE)));
            }
            if (doubt && !unsure) {
                // those left that may come before the last one, to the lanes behind the chosen ones
                int n = top_k;
                const float lo = number(last) - (by_score ? 2.0f * delta + 0x1p-18f * fabsf(number(last)) : 0.0f);
#pragma unroll 1
                for (int i = 0; i < PER; ++i) {
                    // (the lane's best, and those that move up behind it)
                    const int k = key[0], e = (PLACE - (k & PLACE)) * 32 + lane;
                    const bool may = k != NONE && (by_score ? number(mine[e + (e >> 5)]) >= lo : (k & ~PLACE) >= (last & ~PLACE));
                    for (unsigned left = __ballot_sync(ALL, may); left != 0; left &= left - 1, ++n) {
                        const int from = __shfl_sync(ALL, e, __ffs(left) - 1);
                        if (lane == n) id = from;
                    }
#pragma unroll
                    for (int j = 0; j + 1 < PER; ++j) key[j] = key[j + 1];
                    key[PER - 1] = NONE;
                }
                __syncwarp();
                if (n <= 32)
                    id = rank64(a, t, id, n, mine, lane);
                else
                    unsure = true;
            }
        }
        if (unsure) id = choose64(a, t, shared[warp], lane);
        // the weights
        float v = 0.0f, w = 0.0f;
        if (lane < top_k) {
            v = logit(a, t, id);
            w = softmax ? expf(v - top) / sum : 1.0f / (1.0f + expf(-v));
        }
        if (d.normalize) {
            // Scores that FP32 holds badly or not at all (e^-87 is 2^-126) still have ratios: in units of e^most, most the
            // largest chosen logit (with sigmoid scores, if that is below 0)
            if (__any_sync(ALL, lane < top_k && (softmax ? v - top : v) < -80.0f)) {
                float most = number(__reduce_max_sync(ALL, lane < top_k ? ordered(v) : NONE));
                if (!softmax) most = fminf(most, 0.0f);  // (of a NaN: 0)
                if (lane < top_k && (softmax || v < 0.0f))
                    w = softmax ? (sum == sum ? expf(v - most) : sum) : expf(v - most) / (1.0f + expf(v));
            }
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

template <int PER, bool FULL>
cudaError_t launch_full(const RouteArgs& a, int num_sms, cudaStream_t st) {
    const int64_t blocks = (a.d.T + RW - 1) / RW;
    route_kernel<PER, FULL><<<static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(num_sms) * (PER == 16 ? 2 : 3))), RW * 32, 0, st>>>(a);
    return cudaGetLastError();
}
template <int PER>
cudaError_t launch(const RouteArgs& a, int num_sms, cudaStream_t st) {
    return a.d.E == PER * 32 ? launch_full<PER, true>(a, num_sms, st) : launch_full<PER, false>(a, num_sms, st);
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
