// gelu.cuh -- GELU to FP32 accuracy, in its left tail too.
#pragma once
#include "ptx.cuh"

namespace g13 {
namespace {

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

}  // namespace
}  // namespace g13
