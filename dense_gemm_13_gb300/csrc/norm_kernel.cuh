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
// Rows that do not start on 16 bytes: where those of all arrays are off by the same number of elements (as in
// contiguous tensors with an odd number of columns), a row's chunks begin that much before its first
// column, so that loads and stores stay whole ("phased"); other rows go element by element, neighbouring lanes on
// neighbouring elements.
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
__device__ __forceinline__ void ld16(const void* p, uint32_t* v, bool on) {  // (else v keeps what it holds)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])
                 : "l"(p), "r"(static_cast<int>(on)));
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

// One thread's part of a row: TPR threads a row, U chunks of 8 elements each.  XT: the 16-bit type of x and the residual, or
// ANY (chosen while the kernel runs, for each chunk, which the compiler turns into both conversions and a choice).
constexpr int ANY = -1;
template <bool F8, int LAY, int XT, int TPR>
struct Part {
    static constexpr bool VEC = LAY != SINGLES;
    static constexpr int W = XT == ANY ? 8 : 4;  // words that hold a chunk
    const NormArgs& a;
    const NormShape& s;
    int t;  // this thread within the row
    int o;  // the row's phase

    __device__ __forceinline__ int col(int u, int i) const {
        return VEC ? (u * TPR + t) * 8 + i - (LAY == PHASED ? o : 0) : (u * 8 + i) * TPR + t;
    }
    __device__ __forceinline__ int x_type() const { return XT == ANY ? a.d.dtype : XT; }
    __device__ __forceinline__ int r_type() const { return XT == ANY ? a.d.residual_dtype : XT; }
    __device__ __forceinline__ bool in(int c) const { return static_cast<unsigned>(c) < static_cast<unsigned>(s.cols); }
    __device__ __forceinline__ bool whole(int u) const {
        return VEC && (LAY != PHASED || col(u, 0) >= 0) && col(u, 0) + 8 <= s.cols;
    }

    // Chunks past the row's end cost a branch only (one by one each took some 200 instructions: 4000 x 2049, 26 us).
    __device__ __forceinline__ bool none(int u) const { return col(u, 0) >= s.cols; }

    // The raw elements of chunk u of the row that begins at element `at` of p; zeros where the row has none.
    template <typename T>
    __device__ __forceinline__ void singles(const T* p, int u, Raw8<W>& r) const {
#pragma unroll
        for (int i = 0; i < W; ++i) r.v[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = in(col(u, i)) ? p[col(u, i)] : T(0);
            if (sizeof(T) == 4)
                r.v[i % W] = v;
            else
                r.v[i / 2] |= v << i % 2 * 16;
        }
    }
    __device__ __forceinline__ void singles(const void* p, int type, int64_t at, int u, Raw8<W>& r) const {
        if (W == 8 && type == GEMM_F32)
            singles(static_cast<const uint32_t*>(p) + at, u, r);
        else
            singles(static_cast<const uint16_t*>(p) + at, u, r);
    }
    // Whether chunk u takes wide loads: in phased rows what is in it besides the row's elements then lies between the array's first and
    // last element, in the gap between rows or in the next row, and is left out afterwards.
    __device__ __forceinline__ bool wide(int64_t row, int64_t ld, int u) const {
        const int c = col(u, 0);
        if (LAY != PHASED) return whole(u);
        return c < s.cols && (c >= 0 || row * ld >= 8) && (c + 8 <= s.cols || (s.rows - 1 - row) * ld >= 8);
    }
    // (A predicate instead of a branch, behind which the loaded values are copied, and waited for: FP16 with an FP32
    // residual, 4000 x 2560, 23 -> 19 us.  Of 16-bit rows alone the branch is kept: 8192 x 8192, 87.5 us, else 90.)
    __device__ __forceinline__ void load(const void* p, int type, int64_t row, int64_t ld, int u, Raw8<W>& r) const {
        if constexpr (!VEC) {
            singles(p, type, row * ld, u, r);
        } else {
            const bool four = W == 8 && type == GEMM_F32, on = wide(row, ld, u);
            const char* c = static_cast<const char*>(p) + (row * ld + col(u, 0)) * (four ? 4 : 2);
            if constexpr (LAY == ALIGNED && W == 4) {
                if (on) ld16(c, r.v);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) r.v[i] = 0;
                ld16(c, r.v, on);
                if (W == 8) ld16(c + 16, r.v + 4 % W, on && four);
            }
        }
    }
    // The numbers of a chunk that was loaded, those past the row's ends zero.
    __device__ __forceinline__ void numbers(const void* p, int type, int64_t row, int64_t ld, int u, const Raw8<W>& r,
                                            float (&v)[8]) const {
        if (!VEC || whole(u) || wide(row, ld, u)) {
            to_floats(type, r, v);
        } else if (none(u)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        } else {
            Raw8<W> q;
            singles(p, type, row * ld, u, q);
            to_floats(type, q, v);
        }
        if (LAY == PHASED && !whole(u)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = in(col(u, i)) ? v[i] : 0.0f;
        }
    }
    // Numbers to chunk u of the row that begins at element `at` of p, rounded to its type.
    __device__ __forceinline__ void store(void* p, int type, int64_t at, int u, const float (&v)[8]) const {
        if (none(u)) return;
        if (!whole(u)) {
            if (type == GEMM_F32) {
                float* q = static_cast<float*>(p) + at;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (in(col(u, i))) q[col(u, i)] = v[i];
            } else {
                uint16_t* q = static_cast<uint16_t*>(p) + at;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t two = pack16(type, v[i], v[i + 1]);
                    if (in(col(u, i))) q[col(u, i)] = static_cast<uint16_t>(two);
                    if (in(col(u, i + 1))) q[col(u, i + 1)] = static_cast<uint16_t>(two >> 16);
                }
            }
        } else if (type == GEMM_F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at + col(u, 0));
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at + col(u, 0)) =
                make_uint4(pack16(type, v[0], v[1]), pack16(type, v[2], v[3]), pack16(type, v[4], v[5]),
                           pack16(type, v[6], v[7]));
        }
    }

    // v = h of chunk u (zeros where the row has none); writes h.
    __device__ __forceinline__ void sum_up(int64_t row, int u, const Raw8<W>& rx, const Raw8<W>& rr, float (&v)[8],
                                           bool write) const {
        const gemm_norm_desc_t& d = a.d;
        numbers(a.x, x_type(), row, d.ldx, u, rx, v);
        if (!a.r) return;
        float w[8];
        numbers(a.r, r_type(), row, d.ldr, u, rr, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
        if (W == 4 || r_type() != GEMM_F32) {
            Raw8<W> h{};
#pragma unroll
            for (int i = 0; i < 4; ++i) h.v[i] = pack16(r_type(), v[2 * i], v[2 * i + 1]);
            to_floats(r_type(), h, v);
        }
        if (write) store(a.h, r_type(), row * d.ldh, u, v);
    }

    // The weight of chunk u, its offset added.
    __device__ __forceinline__ void weight(int u, float (&w)[8]) const {
        const gemm_norm_desc_t& d = a.d;
        const int c = col(u, 0);
        if (!a.w || none(u)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        } else if (LAY == ALIGNED && whole(u)) {
            Raw8<8> rw;
            const char* p = static_cast<const char*>(a.w) + c * (d.weight_dtype == GEMM_F32 ? 4 : 2);
            const uint4 lo = __ldg(reinterpret_cast<const uint4*>(p));
            rw.v[0] = lo.x, rw.v[1] = lo.y, rw.v[2] = lo.z, rw.v[3] = lo.w;
            if (d.weight_dtype == GEMM_F32) {
                const uint4 hi = __ldg(reinterpret_cast<const uint4*>(p) + 1);
                rw.v[4] = hi.x, rw.v[5] = hi.y, rw.v[6] = hi.z, rw.v[7] = hi.w;
            }
            to_floats(d.weight_dtype, rw, w);
        } else if (LAY == PHASED && s.wide_weight && c + o + 8 <= s.cols) {
            // two whole chunks, of which eight 16-bit numbers from the (8 - o)th are the ones
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + c + o);
            const uint4 hi = __ldg(p), lo = o && c >= 0 ? __ldg(p - 1) : hi;  // (c <= 0: there is none before it, nor any need)
            const uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t h[6], k[5];
            Raw8<8> rw;
            const int from = o ? 8 - o : 0;
#pragma unroll
            for (int i = 0; i < 6; ++i) h[i] = from & 4 ? q[i + 2] : q[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) k[i] = from & 2 ? h[i + 1] : h[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) rw.v[i] = __funnelshift_r(k[i], k[i + 1], from % 2 * 16);
            to_floats(d.weight_dtype, rw, w);
        } else if (d.weight_dtype == GEMM_F32) {
            const float* p = static_cast<const float*>(a.w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = in(col(u, i)) ? __ldg(p + col(u, i)) : 0.0f;
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(a.w);
            uint32_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = in(col(u, i)) ? __ldg(p + col(u, i)) : 0u;
            Raw8<8> rw;
#pragma unroll
            for (int i = 0; i < 4; ++i) rw.v[i] = e[2 * i] | e[2 * i + 1] << 16;
            to_floats(d.weight_dtype, rw, w);
        }
        if (d.weight_offset != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] += d.weight_offset;
        }
    }
    // v (rs + rs_lo) w to 2^-46 of itself, rounded to odd (the last bit set where something was cut off), so that the
    // rounding to four bits that follows does not see a tie that is none.  (v rs first: it is at most the root of the row's
    // length, while v w may lie beyond FP32 where the result does not.)
    static __device__ __forceinline__ float to_odd(float v, float w, float rs, float rs_lo) {
        const float p = v * rs, p_lo = fmaf(v, rs_lo, fmaf(v, rs, -p)), c = p_lo * w, hi = fmaf(p, w, c);
        const float lo = fmaf(p, w, -hi) + c;
        int bits = __float_as_int(hi);
        if (lo != 0.0f && fabsf(hi) < INFINITY && (bits & 1) == 0) bits += (lo < 0.0f) == (hi < 0.0f) ? 1 : -1;
        return hi == 0.0f ? hi : __int_as_float(bits);
    }
    // Whether numbers may round to another E4M3 value if they are off by four units in the last place: next to a tie of
    // the third mantissa bit, or, below 2^-6, where E4M3's values are 2^-9 apart, of that after 2^-6 is added.
    struct Doubt {
        uint32_t tie = 0xFFFFFFFFu;
        __device__ __forceinline__ void see(float y) {  // the lowest 20 bits, counted from four before a tie
            tie = min(tie, __float_as_uint(y) * 4096u + ((4u - 0x80000u) << 12));
        }
        __device__ __forceinline__ void see_low(float y) {
            if (fabsf(y) < 0.015625f) see(fabsf(y) + 0.015625f);
        }
        __device__ __forceinline__ bool any() const { return tie < (8u << 12); }
    };
    // Whether one of four E4M3 codes is below 2^-5.
    static __device__ __forceinline__ bool low(uint32_t codes) {
        return (((codes & 0x70707070u) + 0x7F7F7F7Fu) & 0x80808080u) != 0x80808080u;
    }
    // Whether a block's largest may be on the other side of 1.75.
    static __device__ __forceinline__ bool near_border(uint32_t top) { return ((top + 4u - 0x600000u) & 0x7FFFFFu) < 9u; }

    // y of chunk u from its h: rs (+ rs_lo) is the row's factor.
    __device__ __forceinline__ void finish(int64_t row, int u, const float (&v)[8], float rs, float rs_lo) const {
        const gemm_norm_desc_t& d = a.d;
        float w[8], y[8];
        if (!F8 && none(u)) return;
        weight(u, w);
        const float r1 = rs + rs_lo;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * r1 * w[i];
        if constexpr (!F8) {
            store(a.y, d.out_dtype, row * d.ldy, u, y);
        } else {
            // (every lane of the warp is here: rows of a warp end together, at rows_all)
            const int lane = threadIdx.x & 31;
            uint8_t* codes = static_cast<uint8_t*>(a.y) + row * s.row_bytes;
            uint8_t* tile = a.scales + (row >> 7) * s.col_tiles * kFp4TileBytes + (row & 31) * 16 + (row >> 5 & 3) * 4;
            const bool live = row < s.rows;
            // Three roundings put y off by less than four units in its last place.  Where that may matter to a value of
            // the warp (one warp in a few hundred), all of its values are worked out again, exactly.
            if constexpr (VEC) {
                uint32_t byte = 0, c0, c1;
                for (bool again = false;; again = true) {
                    uint32_t top = 0;
                    if (!whole(u)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = in(col(u, i)) ? y[i] : 0.0f;  // (a factor of NaN leaves the padding zero)
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    byte = mxfp8_scale(top);
                    const float inv = ue8m0_value(254u - min(byte, 254u));
                    Doubt doubt;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] *= inv;
                        doubt.see(y[i]);
                    }
                    c0 = e4m3x4(y), c1 = e4m3x4(y + 4);
                    if (again) break;
                    if (low(c0) || low(c1)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) doubt.see_low(y[i]);
                    }
                    if (!__any_sync(0xFFFFFFFFu, doubt.any() || near_border(top))) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = to_odd(v[i], w[i], rs, rs_lo);
                }
                if (live && col(u, 0) < s.row_bytes)
                    *reinterpret_cast<uint2*>(codes + col(u, 0)) = make_uint2(c0, c1);
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
                    Doubt doubt;
                    bool border = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        byte[i] = mxfp8_scale(top[i]);
                        scaled[i] = y[i] * ue8m0_value(254u - min(byte[i], 254u));
                        doubt.see(scaled[i]);
                        doubt.see_low(scaled[i]);
                        border = border || near_border(top[i]);
                    }
                    if (again || !__any_sync(0xFFFFFFFFu, doubt.any() || border)) break;
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

// A thread's sum of squares in FP32: in one number, or (Two) in two with the roundings' errors beside it (D. E. Knuth's
// two-sum), the even and the odd elements side by side in packed instructions: the sum is then exact but for some 2^-40 of it.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
template <bool TWO, bool EXACT>  // EXACT: the squares are (those of 16-bit numbers)
struct Squares {
    uint64_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t x = pack2(v[i], v[i + 1]), p = fma2(x, x, 0);
            const uint64_t s = add2(hi, p), t = sub2(s, hi), e = add2(sub2(hi, sub2(s, t)), sub2(p, t));
            lo = add2(lo, e);
            if (!EXACT) lo = add2(lo, fma2(x, x, p ^ 0x8000000080000000ull));
            hi = s;
        }
    }
    __device__ __forceinline__ Two sum() const;
};
template <bool EXACT>
struct Squares<false, EXACT> {
    float acc = 0.0f;
    __device__ __forceinline__ void add(const float (&v)[8]) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(v[i], v[i], q);
        acc += q;
    }
    __device__ __forceinline__ float sum() const { return acc; }
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
template <bool TWO, bool EXACT>
__device__ __forceinline__ Two Squares<TWO, EXACT>::sum() const {
    const float2 h = unpack2(hi), l = unpack2(lo);
    // (an infinite or NaN sum has no error beside it)
    return g13::add(Two{h.x, fabsf(h.x) < INFINITY ? l.x : 0.0f}, Two{h.y, fabsf(h.y) < INFINITY ? l.y : 0.0f});
}
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

// The sum over the warp of numbers >= 0 (none of them -0 or below): as integers in units of 2^-24 of the largest's binade
// and 2^-25 of that, by integer reductions of the warp, exact but for 2^-49 of the largest (five steps of shuffles with
// `add` are 70 instructions; these are 25).
__device__ __forceinline__ Two warp_sum(Two v) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v.hi));
    if (top >= 0x7F800000u) return Two{__uint_as_float(top), 0.0f};  // an infinity or a NaN
    const uint32_t e = max(top >> 23, 25u);
    const float scale = __uint_as_float((278u - e) << 23), unit = __uint_as_float((e - 24u) << 23);
    const float h = v.hi * scale;  // below 2^25: 32 of them are below 2^30 (and the rests, one at most, in units of 2^-25)
    const int i = __float2int_rn(h);
    const int j = __float2int_rn(fmaf(v.lo, scale, h - __int2float_rn(i)) * 0x1p25f);
    const int si = __reduce_add_sync(0xFFFFFFFFu, i), sj = __reduce_add_sync(0xFFFFFFFFu, j);
    const float hi = __int2float_rn(si);
    const float lo = fmaf(__int2float_rn(sj), 0x1p-25f, __int2float_rn(si - __float2int_rn(hi)));
    const float all = hi + lo;
    return Two{all * unit, (lo - (all - hi)) * unit};
}

template <typename S>
__device__ __forceinline__ S shuffle_sum(S v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v = add(v, from_lane(v, o));
    return v;
}

// CTAs per SM that the registers are kept for: a thousand threads, fewer where a thread holds more.
__host__ __device__ constexpr int norm_ctas(int lay, int xt, int tpr, int u) {
    const int threads = u == 4 ? 512 : u == 3 || (lay != SINGLES && xt == ANY && u == 2) ? 768 : 1024;
    return threads / (tpr < 128 ? 128 : tpr);
}

// U = 0: the row is read twice instead of kept.
template <bool F8, int LAY, int XT, int TPR, int U>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, norm_ctas(LAY, XT, TPR, U)) rms_norm_kernel(const NormArgs a, const NormShape s) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR;
    constexpr int RPC = THREADS / TPR;  // rows of a CTA at a time
    constexpr int WARPS = TPR / 32;
    using S = typename std::conditional<F8, Two, float>::type;
    constexpr int LANES = WARPS <= 2 ? 2 : WARPS <= 4 ? 4 : WARPS <= 8 ? 8 : WARPS <= 16 ? 16 : 32;  // that hold their sums
    // In mxfp8 blocks begin at column 0: a phased row's h goes through shared memory to threads that hold it as an
    // aligned row (a word more after each 32, so that neither side's lanes, eight words apart, meet in a bank).
    constexpr bool MOVE = F8 && LAY == PHASED;
    constexpr int MOVE_ROW = TPR * U * 8 / 32 * 33;
    __shared__ float moved[MOVE ? RPC * MOVE_ROW : 1];
    __shared__ S partial[2][THREADS / 32];
    const int slot = threadIdx.x / TPR;
    using P = Part<F8, LAY, XT, TPR>;
    constexpr int W = P::W;
    P p{a, s, static_cast<int>(threadIdx.x) % TPR, 0};
    const gemm_norm_desc_t& d = a.d;
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPC; base < s.rows_all;
         base += static_cast<int64_t>(gridDim.x) * RPC, turn ^= 1) {
        const int64_t row = base + slot;
        const int64_t row_in = min(row, s.rows - 1);  // rows of the padding read the last one again
        const bool live = row < s.rows;
        if (LAY == PHASED) p.o = (s.phase + static_cast<int>(row_in & 7) * s.phase_step) & 7;
        Squares<F8, XT != ANY> squares;
        const auto load = [&](int u, Raw8<W>& rx, Raw8<W>& rr) {
            p.load(a.x, p.x_type(), row_in, d.ldx, u, rx);
            if (a.r) p.load(a.r, p.r_type(), row_in, d.ldr, u, rr);
        };
        float v[U > 0 ? U : 1][8];
        if constexpr (U > 0) {
            Raw8<W> rx[U], rr[U];
            // (all loads before the first store, which they would wait for: an output may be an input's own array)
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, rx[u], rr[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p.sum_up(row_in, u, rx[u], rr[u], v[u], a.h != nullptr && live);
                squares.add(v[u]);
                if constexpr (MOVE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = (u * TPR + p.t) * 8 + i;
                        moved[slot * MOVE_ROW + at + (at >> 5)] = v[u][i];
                    }
                }
            }
        } else {
            for (int u = 0; p.col(u, 0) < s.cols; ++u) {
                Raw8<W> rx, rr;
                load(u, rx, rr);
                p.sum_up(row_in, u, rx, rr, v[0], a.h != nullptr && live);
                squares.add(v[0]);
            }
        }
        S sum;
        if constexpr (F8 && TPR >= 32)
            sum = warp_sum(squares.sum());
        else
            sum = shuffle_sum(squares.sum(), TPR < 32 ? TPR : 32);
        if constexpr (WARPS > 1) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) partial[turn][threadIdx.x >> 5] = sum;
            __syncthreads();  // (the other buffer's readers have passed the barrier before)
            sum = lane < WARPS ? partial[turn][slot * WARPS + lane] : S{};
            if constexpr (F8)
                sum = warp_sum(sum);
            else
                sum = broadcast(shuffle_sum(sum, LANES));
        } else if (MOVE) {
            __syncwarp();
        }
        float rs, rs_lo;
        factor(sum, s.inv, d.eps, rs, rs_lo);
        if constexpr (MOVE) {
            const Part<F8, ALIGNED, XT, TPR> q{a, s, p.t, 0};
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = q.col(u, i) + p.o;
                    v[u][i] = q.in(q.col(u, i)) ? moved[slot * MOVE_ROW + at + (at >> 5)] : 0.0f;
                }
                q.finish(row, u, v[u], rs, rs_lo);
            }
            if (WARPS > 1)  // before the next row's h comes there
                __syncthreads();
            else
                __syncwarp();
        } else if constexpr (U > 0) {
            if (F8 || live) {
#pragma unroll
                for (int u = 0; u < U; ++u) p.finish(row, u, v[u], rs, rs_lo);
            }
        } else if (F8 || live) {
            // every lane of a warp takes as many turns, past the padding of the codes and the scales
            const int64_t end = F8 ? s.col_tiles * 128 : s.cols;
            for (int u = 0; static_cast<int64_t>(u) * TPR * 8 < end; ++u) {
                Raw8<W> rx, rr;
                if (a.h) {  // what this thread wrote in the first turn
                    p.load(a.h, p.r_type(), row_in, d.ldh, u, rx);
                    p.numbers(a.h, p.r_type(), row_in, d.ldh, u, rx, v[0]);
                } else {
                    load(u, rx, rr);
                    p.sum_up(row_in, u, rx, rr, v[0], false);
                }
                p.finish(row, u, v[0], rs, rs_lo);
            }
        }
    }
}

template <bool F8, int LAY, int XT, int TPR, int U>
cudaError_t launch(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR, RPC = THREADS / TPR;
    const int64_t blocks = (s.rows_all + RPC - 1) / RPC;
    const int64_t grid = std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * norm_ctas(LAY, XT, TPR, U));
    rms_norm_kernel<F8, LAY, XT, TPR, U><<<static_cast<unsigned>(grid), THREADS, 0, st>>>(a, s);
    return cudaGetLastError();
}

template <bool F8, int LAY, int XT>
cudaError_t launch_shape(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    // what a row's threads hold: all of its codes' and scales' padding too, and the columns before a phased row's first
    const int64_t codes = F8 ? (LAY == SINGLES ? s.col_tiles * 128 : (s.cols + 31) / 32 * 32) : 0;
    const int64_t chunks = (std::max<int64_t>(s.cols + (LAY == PHASED ? 7 : 0), codes) + 7) / 8;
    if constexpr (LAY == SINGLES) {
        if (chunks <= 32) return launch<F8, LAY, XT, 32, 1>(a, s, num_sms, st);
        if (chunks <= 128) return launch<F8, LAY, XT, 64, 2>(a, s, num_sms, st);
        if (chunks <= 512) return launch<F8, LAY, XT, 256, 2>(a, s, num_sms, st);
        if (chunks <= 2048) return launch<F8, LAY, XT, 512, 4>(a, s, num_sms, st);
        return launch<F8, LAY, XT, 512, 0>(a, s, num_sms, st);
    } else {
        if (chunks <= 8) return launch<F8, LAY, XT, 8, 1>(a, s, num_sms, st);
        if (chunks <= 16) return launch<F8, LAY, XT, 16, 1>(a, s, num_sms, st);
        if (chunks <= 32) return launch<F8, LAY, XT, 32, 1>(a, s, num_sms, st);
        if constexpr (LAY == ALIGNED) {
            if (chunks > 2048) return launch<F8, LAY, XT, 512, 0>(a, s, num_sms, st);
            // one chunk a thread where there are few rows: latency counts
            if (s.rows <= 2 * num_sms) {
                if (chunks <= 64) return launch<F8, LAY, XT, 64, 1>(a, s, num_sms, st);
                if (chunks <= 128) return launch<F8, LAY, XT, 128, 1>(a, s, num_sms, st);
                if (chunks <= 256) return launch<F8, LAY, XT, 256, 1>(a, s, num_sms, st);
                if (chunks <= 512) return launch<F8, LAY, XT, 512, 1>(a, s, num_sms, st);
                if (chunks <= 768) return launch<F8, LAY, XT, 768, 1>(a, s, num_sms, st);
                if (chunks <= 1024) return launch<F8, LAY, XT, 1024, 1>(a, s, num_sms, st);
            }
        }
        if (chunks <= 64) return launch<F8, LAY, XT, 32, 2>(a, s, num_sms, st);
        if (chunks <= 96) return launch<F8, LAY, XT, 32, 3>(a, s, num_sms, st);
        if (chunks <= 128) return launch<F8, LAY, XT, 64, 2>(a, s, num_sms, st);
        if (chunks <= 192) return launch<F8, LAY, XT, 64, 3>(a, s, num_sms, st);
        if (chunks <= 256) return launch<F8, LAY, XT, 128, 2>(a, s, num_sms, st);
        if (chunks <= 384) return launch<F8, LAY, XT, 128, 3>(a, s, num_sms, st);
        if (chunks <= 512) return launch<F8, LAY, XT, 256, 2>(a, s, num_sms, st);
        if (chunks <= 768) return launch<F8, LAY, XT, 256, 3>(a, s, num_sms, st);
        if constexpr (F8 && LAY == PHASED)
            return launch<F8, LAY, XT, 512, 2>(a, s, num_sms, st);
        else
            return chunks <= 1024 ? launch<F8, LAY, XT, 512, 2>(a, s, num_sms, st)
                                  : launch<F8, LAY, XT, 512, 4>(a, s, num_sms, st);
    }
}

// One of the files of kernels: rows of a 16-bit type's own, or of any types.
template <bool F8, int XT>
cudaError_t launch_norm_lay(const NormArgs& a, const NormShape& s, int num_sms, cudaStream_t st) {
    if (s.lay == ALIGNED) return launch_shape<F8, ALIGNED, XT>(a, s, num_sms, st);
    if (s.lay == PHASED) return launch_shape<F8, PHASED, XT>(a, s, num_sms, st);
    return launch_shape<F8, SINGLES, XT>(a, s, num_sms, st);
}

}  // namespace
}  // namespace g13
