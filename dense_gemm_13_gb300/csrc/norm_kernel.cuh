// norm_kernel.cuh -- root-mean-square norm of rows, with the residual's addition before it and
// an output in 16 or 32 bits or in mxfp8:
//
//   h = cast(x + r)      (r's type; without r: h = x)
//   y = h / sqrt(mean(h^2) + eps) * (w + offset)
//
// Every element is read once and written once, so memory bounds it: a row stays in its
// threads' registers between the sum and the output (up to 16384 columns; longer rows are
// read a second time, from L2 mostly).  A row belongs to 8, 16 or 32 lanes, or to a CTA, of
// which each thread holds one to four chunks of eight neighbouring elements; the row's sum is
// joined by shuffles, and between warps through shared memory with one barrier.  CTAs are
// persistent, so that one row's loads overlap another's sums on the same SM.
// Rows that are not 16-byte aligned go element by element, neighbouring lanes on neighbouring
// elements.
//
// In mxfp8 four threads' chunks (a warp's 32 elements, where rows are not aligned) are a
// block: its largest magnitude by shuffles, eight codes as one store.  Codes and scales are those of
// the exact y but for what the sum of squares is off by: the threads' sums and 1 / sqrt are kept in two
// FP32 numbers each (a few FP64 operations a row would take 5 us), and values next to a border are
// worked out again with theirs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "internal.h"
#include "norm.h"

namespace g13 {
namespace {

// A chunk of eight elements as it was loaded: 16-bit types fill the first four words (W = 4: there are no others).
template <int W>
struct Raw8 {
    uint32_t v[W];
};
// (Not through the read-only path: an output may be an input's own array.)
__device__ __forceinline__ void ld16(const void* p, uint32_t* v) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "l"(p));
}
__device__ __forceinline__ float one(const void* p, int type, int64_t i) {
    if (type == GEMM_F32) return static_cast<const float*>(p)[i];
    if (type == GEMM_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void put(void* p, int type, int64_t i, float v) {
    if (type == GEMM_F32)
        static_cast<float*>(p)[i] = v;
    else if (type == GEMM_BF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}
// v as a number of `type`.
__device__ __forceinline__ float round_to(int type, float v) {
    if (type == GEMM_F32) return v;
    if (type == GEMM_BF16) return __bfloat162float(__float2bfloat16_rn(v));
    return __half2float(__float2half_rn(v));
}
template <int W>
__device__ __forceinline__ void to_floats(int type, const Raw8<W>& r, float (&f)[8]) {
    if (W == 8 && type == GEMM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i % W]);
    } else if (type == GEMM_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(r.v[i] << 16);
            f[2 * i + 1] = __uint_as_float(r.v[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&r.v[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}
__device__ __forceinline__ uint32_t pack16(int type, float a, float b) {
    if (type == GEMM_BF16) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&t);
    }
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// One thread's part of a row: TPR threads a row, U chunks of 8 elements each.  With VEC a
// chunk is eight neighbours, else elements TPR apart.
template <bool F8, bool VEC, int W, int TPR>
struct Part {
    const NormArgs& a;
    const NormShape& s;
    int t;  // this thread within the row

    __device__ __forceinline__ int col(int u, int i) const {
        return VEC ? (u * TPR + t) * 8 + i : (u * 8 + i) * TPR + t;
    }
    __device__ __forceinline__ int64_t size(int type) const { return type == GEMM_F32 ? 4 : 2; }

    // The raw elements of chunk u of a row of p (whole chunks of VEC rows only).
    __device__ __forceinline__ void load(const void* p, int type, int64_t at, Raw8<W>& r) const {
        const char* c = static_cast<const char*>(p) + at * (W == 4 ? 2 : size(type));
        ld16(c, r.v);
        if (W == 8 && type == GEMM_F32) ld16(c + 16, r.v + 4 % W);
    }
    __device__ __forceinline__ bool whole(int u) const { return VEC && col(u, 0) + 8 <= s.cols; }
    // The elements of a chunk one by one, as FP32 (zeros past the row's end).  The types are asked once a chunk, and
    // nothing is stored between the loads, which would wait for one another (1000 x 4097: 28.5 us).
    template <typename T>
    __device__ __forceinline__ void singles(const void* p, int64_t at, int u, Raw8<8>& o) const {
        const T* q = static_cast<const T*>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o.v[i] = col(u, i) < s.cols ? __float_as_uint(static_cast<float>(q[col(u, i)])) : 0u;
    }
    __device__ __forceinline__ void singles(const void* p, int type, int64_t at, int u, Raw8<8>& o) const {
        if (type == GEMM_F32)
            singles<float>(p, at, u, o);
        else if (type == GEMM_BF16)
            singles<__nv_bfloat16>(p, at, u, o);
        else
            singles<__half>(p, at, u, o);
    }
    __device__ __forceinline__ void singles(int64_t row, int u, Raw8<8>& rx, Raw8<8>& rr) const {
        singles(a.x, a.d.dtype, row * a.d.ldx, u, rx);
        if (a.r) singles(a.r, a.d.residual_dtype, row * a.d.ldr, u, rr);
    }

    // v = h of chunk u (zeros past the row's end), from raw elements where the chunk is whole; writes h.
    __device__ __forceinline__ void sum_up(int64_t row, int u, const Raw8<W>& rx, const Raw8<W>& rr, float (&v)[8],
                                           bool store) const {
        const gemm_norm_desc_t& d = a.d;
        if (whole(u)) {
            to_floats(d.dtype, rx, v);
            if (a.r) {
                float w[8];
                to_floats(d.residual_dtype, rr, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += w[i];
                if (W == 4 || d.residual_dtype != GEMM_F32) {
                    Raw8<W> o{};
#pragma unroll
                    for (int i = 0; i < 4; ++i) o.v[i] = pack16(d.residual_dtype, v[2 * i], v[2 * i + 1]);
                    to_floats(d.residual_dtype, o, v);
                    if (store) *reinterpret_cast<uint4*>(static_cast<char*>(a.h) + (row * d.ldh + col(u, 0)) * 2) =
                        make_uint4(o.v[0], o.v[1], o.v[2], o.v[3]);
                } else if (store) {
                    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.h) + row * d.ldh + col(u, 0));
                    p[0] = make_float4(v[0], v[1], v[2], v[3]);
                    p[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            return;
        }
        Raw8<8> x8, r8;
        if constexpr (VEC)
            singles(row, u, x8, r8);
        else
            x8 = rx, r8 = rr;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = __uint_as_float(x8.v[i]);
            if (a.r) {
                v[i] = round_to(d.residual_dtype, v[i] + __uint_as_float(r8.v[i]));
                if (store && col(u, i) < s.cols) put(a.h, d.residual_dtype, row * d.ldh + col(u, i), v[i]);
            }
        }
    }

    // The weight of chunk u, its offset added.
    __device__ __forceinline__ void weight(int u, float (&w)[8]) const {
        const gemm_norm_desc_t& d = a.d;
        if (!a.w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        } else if (whole(u)) {
            Raw8<8> rw;
            const char* p = static_cast<const char*>(a.w) + col(u, 0) * size(d.weight_dtype);
            const uint4 lo = __ldg(reinterpret_cast<const uint4*>(p));
            rw.v[0] = lo.x, rw.v[1] = lo.y, rw.v[2] = lo.z, rw.v[3] = lo.w;
            if (d.weight_dtype == GEMM_F32) {
                const uint4 hi = __ldg(reinterpret_cast<const uint4*>(p) + 1);
                rw.v[4] = hi.x, rw.v[5] = hi.y, rw.v[6] = hi.z, rw.v[7] = hi.w;
            }
            to_floats(d.weight_dtype, rw, w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = col(u, i) < s.cols ? one(a.w, d.weight_dtype, col(u, i)) : 0.0f;
        }
        if (d.weight_offset != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] += d.weight_offset;
        }
    }
    // v w (rs + rs_lo) to 2^-46 of itself, rounded to odd (the last bit set where something was cut off), so that the
    // rounding to four bits that follows does not see a tie that is none.
    static __device__ __forceinline__ float to_odd(float v, float w, float rs, float rs_lo) {
        const float p = v * w, e = fmaf(v, w, -p), c = fmaf(p, rs_lo, e * rs), hi = fmaf(p, rs, c);  // v w = p + e
        const float lo = fmaf(p, rs, -hi) + c;
        int bits = __float_as_int(hi);
        if (lo != 0.0f && fabsf(hi) < INFINITY && (bits & 1) == 0) bits += (lo < 0.0f) == (hi < 0.0f) ? 1 : -1;
        return hi == 0.0f ? hi : __int_as_float(bits);
    }
    // Whether a number may round otherwise to three mantissa bits (or, of a block's largest, fall on the other side of
    // 1.75) if it is off by four units in its last place.
    static __device__ __forceinline__ bool near_tie(float y) {
        return ((__float_as_uint(y) + 4u - 0x80000u) & 0xFFFFFu) < 8u;
    }
    static __device__ __forceinline__ bool near_border(uint32_t top) { return ((top + 4u - 0x600000u) & 0x7FFFFFu) < 9u; }

    // y of chunk u from its h: rs (+ rs_lo) is the row's factor.
    __device__ __forceinline__ void finish(int64_t row, int u, const float (&v)[8], float rs, float rs_lo) const {
        const gemm_norm_desc_t& d = a.d;
        float w[8], y[8];
        weight(u, w);
        const float r1 = rs + rs_lo;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * r1 * w[i];
        if constexpr (!F8) {
            if (whole(u)) {
                char* p = static_cast<char*>(a.y) + (row * d.ldy + col(u, 0)) * size(d.out_dtype);
                if (d.out_dtype == GEMM_F32) {
                    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
                    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
                } else {
                    *reinterpret_cast<uint4*>(p) =
                        make_uint4(pack16(d.out_dtype, y[0], y[1]), pack16(d.out_dtype, y[2], y[3]),
                                   pack16(d.out_dtype, y[4], y[5]), pack16(d.out_dtype, y[6], y[7]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col(u, i) < s.cols) put(a.y, d.out_dtype, row * d.ldy + col(u, i), y[i]);
            }
        } else {
            // (every lane of the warp is here: rows of a warp end together, at rows_all)
            const int lane = threadIdx.x & 31;
            uint8_t* codes = static_cast<uint8_t*>(a.y) + row * s.row_bytes;
            uint8_t* tile = a.scales + (row >> 7) * s.col_tiles * kFp4TileBytes + (row & 31) * 16 + (row >> 5 & 3) * 4;
            const bool live = row < s.rows;
            // Three roundings put y off by less than four units in its last place.  Where that may matter to a value of
            // the warp (one warp in a few hundred), all of its values are worked out again, exactly.
            if constexpr (VEC) {
                uint32_t byte = 0;
                for (bool again = false;; again = true) {
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (col(u, i) >= s.cols) y[i] = 0.0f;  // (a factor of NaN leaves the padding zero)
                        top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                    }
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    byte = mxfp8_scale(top);
                    const float inv = ue8m0_value(254u - min(byte, 254u));
                    bool near = near_border(top);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] *= inv;
                        near = near || near_tie(y[i]);
                    }
                    if (again || !__any_sync(0xFFFFFFFFu, near)) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = to_odd(v[i], w[i], rs, rs_lo);
                }
                if (live && col(u, 0) < s.row_bytes)
                    *reinterpret_cast<uint2*>(codes + col(u, 0)) = make_uint2(e4m3x4(y), e4m3x4(y + 4));
                // (a row in the padding, and a block past the row's end: zero.)  Eight lanes have two of a
                // tile's four scales of this row; the first lane of sixteen, or of eight, writes them
                if (!live || col(u, 0) >= s.cols) byte = 0;
                byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
                if constexpr (TPR >= 16) {
                    byte = (byte & 0xFFFFu) | __shfl_down_sync(0xFFFFFFFFu, byte, 8) << 16;
                    if ((lane & 15) == 0 && col(u, 0) / 128 < s.col_tiles)
                        *reinterpret_cast<uint32_t*>(tile + static_cast<int64_t>(col(u, 0) / 128) * kFp4TileBytes) = byte;
                } else {
                    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(tile) = byte & 0xFFFFu;
                }
            } else {
                // (element i of the chunk is in the warp's i-th block of 32 neighbours)
                uint32_t byte[8];
                float scaled[8];
                for (bool again = false;; again = true) {
                    uint32_t top[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (col(u, i) >= s.cols) y[i] = 0.0f;
                        top[i] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                    }
                    bool near = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        byte[i] = mxfp8_scale(top[i]);
                        scaled[i] = y[i] * ue8m0_value(254u - min(byte[i], 254u));
                        near = near || near_tie(scaled[i]) || near_border(top[i]);
                    }
                    if (again || !__any_sync(0xFFFFFFFFu, near)) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = to_odd(v[i], w[i], rs, rs_lo);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = col(u, i), c0 = c & ~31;
                    if (c0 >= s.col_tiles * 128) continue;
                    const float v4[4] = {scaled[i], 0.0f, 0.0f, 0.0f};
                    if (live && c < s.row_bytes) codes[c] = static_cast<uint8_t>(e4m3x4(v4));
                    if (lane == 0)
                        tile[static_cast<int64_t>(c0 / 128) * kFp4TileBytes + (c0 >> 5 & 3)] =
                            static_cast<uint8_t>(live && c0 < s.cols ? byte[i] : 0);
                }
            }
        }
    }
};

// A sum in two FP32 numbers (T. J. Dekker's double length addition, 1971), or in one.
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    float e = (a.hi - (s - t)) + (b.hi - t) + a.lo + b.lo;
    if (!(fabsf(s) < INFINITY)) e = 0.0f;
    const float hi = s + e;
    return Two{hi, fabsf(hi) < INFINITY ? e - (hi - s) : 0.0f};
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float broadcast(float v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ Two broadcast(Two v) { return Two{broadcast(v.hi), broadcast(v.lo)}; }
__device__ __forceinline__ float from_lane(float v, int o) { return __shfl_xor_sync(0xFFFFFFFFu, v, o); }
__device__ __forceinline__ Two from_lane(Two v, int o) { return Two{from_lane(v.hi, o), from_lane(v.lo, o)}; }

// The row's factor 1 / sqrt(sum / cols + eps): rsqrtf's result, and in F8 what it is off by, from the remainder
// 1 - v r^2 (one step of Newton's method).  inv: 1 / cols, in two numbers.
__device__ __forceinline__ void factor(Two sum, Two inv, float eps, float& rs, float& rs_lo) {
    const float m = sum.hi * inv.hi;
    const float m_lo = fmaf(sum.hi, inv.hi, -m) + (sum.hi * inv.lo + sum.lo * inv.hi);
    const Two v = add(Two{m, fabsf(m_lo) < INFINITY ? m_lo : 0.0f}, Two{eps, 0.0f});
    rs = rsqrtf(v.hi);
    const float t = v.hi * rs, t_lo = fmaf(v.hi, rs, -t);
    const float e = fmaf(-t, rs, 1.0f) - t_lo * rs - v.lo * rs * rs;
    rs_lo = fabsf(e) < 1.0f ? 0.5f * rs * e : 0.0f;  // (not for an infinite or NaN sum)
}
__device__ __forceinline__ void factor(float sum, Two inv, float eps, float& rs, float& rs_lo) {
    rs = rsqrtf(sum * inv.hi + eps);
    rs_lo = 0.0f;
}

template <typename S>
__device__ __forceinline__ S shuffle_sum(S v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v = add(v, from_lane(v, o));
    return v;
}

// CTAs per SM that the registers are kept for: a thousand threads, fewer where a thread holds more.
__host__ __device__ constexpr int norm_ctas(bool vec, int w, int tpr, int u) {
    return (u == 4 || (vec && w == 8 && u > 1) ? 512 : u == 3 ? 768 : 1024) / (tpr < 128 ? 128 : tpr);
}

// U = 0: the row is read twice instead of kept.
template <bool F8, bool VEC, int W, int TPR, int U>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, norm_ctas(VEC, W, TPR, U)) rms_norm_kernel(const NormArgs a, const NormShape s) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR;
    constexpr int RPC = THREADS / TPR;  // rows of a CTA at a time
    constexpr int WARPS = TPR / 32;
    using S = typename std::conditional<F8, Two, float>::type;
    constexpr int LANES = WARPS <= 2 ? 2 : WARPS <= 4 ? 4 : WARPS <= 8 ? 8 : WARPS <= 16 ? 16 : 32;  // that hold their sums
    __shared__ S partial[2][THREADS / 32];
    const int slot = threadIdx.x / TPR;
    const Part<F8, VEC, W, TPR> p{a, s, static_cast<int>(threadIdx.x) % TPR};
    const gemm_norm_desc_t& d = a.d;
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPC; base < s.rows_all;
         base += static_cast<int64_t>(gridDim.x) * RPC, turn ^= 1) {
        const int64_t row = base + slot;
        const int64_t row_in = min(row, s.rows - 1);  // rows of the padding read the last one again
        const bool live = row < s.rows;
        float acc = 0.0f;
        const auto square = [&](const float (&v)[8]) {
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) q = fmaf(v[i], v[i], q);
            return q;
        };
        const auto load = [&](int u, Raw8<W>& rx, Raw8<W>& rr) {
            if constexpr (!VEC) p.singles(row_in, u, rx, rr);
            if (!p.whole(u)) return;
            p.load(a.x, d.dtype, row_in * d.ldx + p.col(u, 0), rx);
            if (a.r) p.load(a.r, d.residual_dtype, row_in * d.ldr + p.col(u, 0), rr);
        };
        float v[U > 0 ? U : 1][8];
        if constexpr (U > 0) {
            Raw8<W> rx[U], rr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, rx[u], rr[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p.sum_up(row_in, u, rx[u], rr[u], v[u], a.h != nullptr && live);
                acc += square(v[u]);
            }
        } else {
            for (int u = 0; p.col(u, 0) < s.cols; ++u) {
                Raw8<W> rx, rr;
                load(u, rx, rr);
                p.sum_up(row_in, u, rx, rr, v[0], a.h != nullptr && live);
                acc += square(v[0]);
            }
        }
        S sum = shuffle_sum(S{acc}, TPR < 32 ? TPR : 32);
        if constexpr (WARPS > 1) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) partial[turn][threadIdx.x >> 5] = sum;
            __syncthreads();  // (the other buffer's readers have passed the barrier before)
            sum = broadcast(shuffle_sum(lane < WARPS ? partial[turn][slot * WARPS + lane] : S{}, LANES));
        }
        float rs, rs_lo;
        factor(sum, s.inv, d.eps, rs, rs_lo);
        if constexpr (U > 0) {
            if (F8 || live) {
#pragma unroll
                for (int u = 0; u < U; ++u) p.finish(row, u, v[u], rs, rs_lo);
            }
        } else if (F8 || live) {
            // every lane of a warp takes as many turns, past the padding of the codes and the scales
            const int64_t end = F8 ? s.col_tiles * 128 : s.cols;
            for (int u = 0; static_cast<int64_t>(u) * TPR * 8 < end; ++u) {
                if (a.h) {  // what this thread wrote in the first turn
                    if (p.whole(u)) {
                        Raw8<W> rh;
                        p.load(a.h, d.residual_dtype, row_in * d.ldh + p.col(u, 0), rh);
                        to_floats(d.residual_dtype, rh, v[0]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[0][i] = p.col(u, i) < s.cols ? one(a.h, d.residual_dtype, row_in * d.ldh + p.col(u, i)) : 0.0f;
                    }
                } else {
                    Raw8<W> rx, rr;
                    load(u, rx, rr);
                    p.sum_up(row_in, u, rx, rr, v[0], false);
                }
                p.finish(row, u, v[0], rs, rs_lo);
            }
        }
    }
}

template <bool F8, bool VEC, int W, int TPR, int U>
cudaError_t launch(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR, RPC = THREADS / TPR;
    const int64_t blocks = (s.rows_all + RPC - 1) / RPC;
    const int64_t grid = std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * norm_ctas(VEC, W, TPR, U));
    rms_norm_kernel<F8, VEC, W, TPR, U><<<static_cast<unsigned>(grid), THREADS, 0, st>>>(a, s);
    return cudaGetLastError();
}

template <bool F8, bool VEC, int W>
cudaError_t launch_shape(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    // what a row's threads hold: all of its codes' and scales' padding too
    const int64_t cols = F8 ? (VEC ? (s.cols + 31) / 32 * 32 : s.col_tiles * 128) : s.cols;
    const int64_t chunks = (cols + 7) / 8;
    if (VEC && chunks <= 8) return launch<F8, VEC, W, VEC ? 8 : 32, 1>(a, s, num_sms, st);
    if (VEC && chunks <= 16) return launch<F8, VEC, W, VEC ? 16 : 32, 1>(a, s, num_sms, st);
    if (chunks <= 32) return launch<F8, VEC, W, 32, 1>(a, s, num_sms, st);
    if (chunks > 2048) return launch<F8, VEC, W, 512, 0>(a, s, num_sms, st);
    // one chunk a thread where there are few rows: latency counts
    if (s.rows <= 2 * num_sms) {
        if (chunks <= 64) return launch<F8, VEC, W, 64, 1>(a, s, num_sms, st);
        if (chunks <= 128) return launch<F8, VEC, W, 128, 1>(a, s, num_sms, st);
        if (chunks <= 256) return launch<F8, VEC, W, 256, 1>(a, s, num_sms, st);
        if (chunks <= 512) return launch<F8, VEC, W, 512, 1>(a, s, num_sms, st);
        if (chunks <= 768) return launch<F8, VEC, W, 768, 1>(a, s, num_sms, st);
        if (chunks <= 1024) return launch<F8, VEC, W, 1024, 1>(a, s, num_sms, st);
    }
    if constexpr (!VEC) {  // single elements, eight a chunk: threads without any would cost as much
        if (chunks > 128 && chunks <= 192) return launch<F8, VEC, W, 64, 3>(a, s, num_sms, st);
        if (chunks > 256 && chunks <= 384) return launch<F8, VEC, W, 128, 3>(a, s, num_sms, st);
        if (chunks > 512 && chunks <= 768) return launch<F8, VEC, W, 256, 3>(a, s, num_sms, st);
        if (chunks > 1024 && chunks <= 1536) return launch<F8, VEC, W, 512, 3>(a, s, num_sms, st);
    }
    if (chunks <= 64) return launch<F8, VEC, W, 32, 2>(a, s, num_sms, st);
    if (chunks <= 128) return launch<F8, VEC, W, 64, 2>(a, s, num_sms, st);
    if (chunks <= 256) return launch<F8, VEC, W, 128, 2>(a, s, num_sms, st);
    if (chunks <= 512) return launch<F8, VEC, W, 256, 2>(a, s, num_sms, st);
    if (chunks <= 1024) return launch<F8, VEC, W, 512, 2>(a, s, num_sms, st);
    return launch<F8, VEC, W, 512, 4>(a, s, num_sms, st);
}


// norm.cu and norm8.cu
template <bool F8>
cudaError_t launch_norm_kind(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    const gemm_norm_desc_t& d = a.d;
    const auto on = [&](const void* p, int type, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (d.rows <= 1 || ld * (type == GEMM_F32 ? 4 : 2) % 16 == 0);
    };
    const bool vec = on(a.x, d.dtype, d.ldx) && on(a.r, d.residual_dtype, d.ldr) && on(a.h, d.residual_dtype, d.ldh) &&
                     on(a.w, d.weight_dtype, 0) && (F8 || on(a.y, d.out_dtype, d.ldy));
    if (!vec) return launch_shape<F8, false, 8>(a, s, num_sms, st);
    if (d.dtype == GEMM_F32 || d.residual_dtype == GEMM_F32) return launch_shape<F8, true, 8>(a, s, num_sms, st);
    return launch_shape<F8, true, 4>(a, s, num_sms, st);
}

}  // namespace
}  // namespace g13
