// act_dev.cuh -- activations that more than one kernel evaluates.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// 1 / (1 + exp(-g)) by the hardware's 2^x and reciprocal (2^-22 and one unit in
// the last place), subnormals flushed (0 below -87.3); relative error at most
// (3.5 + |g|) 2^-23, the argument's rounding included: __expf and __fdividef take twice the
// instructions for them, which the epilogues feel (with fewer tests per value:
// gradient of the projections at 1999 tokens 67.7 -> 62.0 us, 8-bit gate/up of
// 65536 rows 1382 -> 1293).
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// v Phi(v), Phi the normal distribution's mass below v.  (1 + erf(v / sqrt 2)) / 2
// cancels for negative v (4% off at -5, zero from -5.6 on), so both sides use
// the tail Q = Phi(-z), z = |v|: v Q below zero, v - v Q above.
//   Q = exp(-z^2 / 2) R(z),  R = erfcx(z / sqrt 2) / 2 = t p(t),  t = 1 / (1 + 0.345 z)
// (the form of Hastings' approximations); p of degree 8 fitted here to R / t on
// [0, 13.4] by iteratively reweighted least squares, relative error 2.0e-8.  The
// exponent's rounding errors, which z^2 / 2 would multiply, are carried along:
//   -z^2 / (2 ln 2) = a + l,  2^(a + l) = 2^a (1 + l ln 2).
// Relative error in units of 2^-23: 2 for the hardware's 2^x; 3.5 for t (1 for
// its reciprocal, half a unit for the argument, times the slope of ln R over
// ln t, up to 2.3); 2.7 for p's coefficients and steps; half a unit each for
// t p, 2^x's correction, Q and the result; 0.2 for the fit: at most 10.4 (3.4
// measured).  A mass below 2^-126 (v < -12.9) keeps fewer digits, none from -13.2 on.
// 16384 x 4096 x 4096 with gelu, bias and residual: 357 us; by erff 348, by
// normcdff, as accurate, 385.  777 ragged rows of 650 x 1160: 19.9, 19.4 and 24.4.
__device__ __forceinline__ float gelu(float v) {
    const float z = fminf(fabsf(v), 14.f);      // (2^x is 0 from 13.3 on)
    float t, e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(z, 0.345f, 1.f)));
    float p = -0.028427263721823692f;
    p = fmaf(p, t, 0.1454882174730301f);
    p = fmaf(p, t, -0.2715703547000885f);
    p = fmaf(p, t, 0.18761830031871796f);
    p = fmaf(p, t, -0.03787045553326607f);
    p = fmaf(p, t, 0.11190465837717056f);
    p = fmaf(p, t, 0.11721377074718475f);
    p = fmaf(p, t, 0.1380240023136139f);
    p = fmaf(p, t, 0.13761912286281586f);
    constexpr float kHi = -0.72134752f, kLo = -9.629815e-9f;   // -1 / (2 ln 2)
    const float s = z * z, a = s * kHi;
    const float l = fmaf(fmaf(z, z, -s), kHi, fmaf(s, kLo, fmaf(s, kHi, -a)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
    const float q = p * t * fmaf(e * l, 0.69314718f, e);
    return v > 0.f ? fmaf(-z, q, v) : v * q;     // (NaN stays)
}

}  // namespace moe
