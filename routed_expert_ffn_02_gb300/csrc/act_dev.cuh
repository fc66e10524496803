// act_dev.cuh -- activations that more than one kernel evaluates.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// The hardware's 2^x (2^-22) and reciprocal (one unit in the last place),
// subnormals flushed.
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + exp(-g)), 0 below -87.3; relative error at most (3.5 + |g|) 2^-23, the
// argument's rounding included.  __expf and __fdividef take twice the
// instructions for them, which the epilogues feel (with fewer tests per value:
// gradient of the projections at 1999 tokens 67.7 -> 62.0 us, 8-bit gate/up of
// 65536 rows 1382 -> 1293).
__device__ __forceinline__ float sigmoid(float g) {
    return rcp(1.0f + ex2(g * -1.4426950408889634f));
}

// Pairs of fp32 values.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 two(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 each(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
// t p, 2^x's correction, Q and the result; 0.2 for the fit: at most 10.4 (4
// measured).  A mass below 2^-126 (v < -12.9) keeps fewer digits, none from -13.2 on.
// Two values at once, by two-wide FMAs: 16384 x 4096 x 4096 with gelu, bias and
// residual 348 us, one at a time 357 (and silu, whose code then lies farther
// apart, 1% slower), by erff 350, by normcdff, as accurate, 385.  777 ragged rows of
// 650 x 1160: 18.6, 19.9, 19.4 and 24.4.
__device__ __forceinline__ void gelu2(float& v0, float& v1) {
    const auto c = [](float v) { return two(v, v); };
    constexpr float kHi = -0.72134752f, kLo = -9.629815e-9f;   // -1 / (2 ln 2)
    const float z0 = fminf(fabsf(v0), 14.f), z1 = fminf(fabsf(v1), 14.f);      // (2^x is 0 from 13.3 on)
    const f32x2 z = two(z0, z1), s = mul2(z, two(-z0, -z1));                   // -z^2
    const float2 d = each(fma2(z, c(0.345f), c(1.f)));
    const f32x2 t = two(rcp(d.x), rcp(d.y));
    f32x2 p = c(-0.028427263721823692f);
    p = fma2(p, t, c(0.1454882174730301f));
    p = fma2(p, t, c(-0.2715703547000885f));
    p = fma2(p, t, c(0.18761830031871796f));
    p = fma2(p, t, c(-0.03787045553326607f));
    p = fma2(p, t, c(0.11190465837717056f));
    p = fma2(p, t, c(0.11721377074718475f));
    p = fma2(p, t, c(0.1380240023136139f));
    p = fma2(p, t, c(0.13761912286281586f));
    const f32x2 na = mul2(s, c(kHi));                                          // -a
    const f32x2 l = fma2(fma2(z, z, s), c(kHi), fma2(s, c(-kLo), fma2(s, c(-kHi), na)));
    const float2 a = each(na);
    const f32x2 e = two(ex2(-a.x), ex2(-a.y));
    const float2 q = each(mul2(mul2(p, t), fma2(mul2(e, l), c(0.69314718f), e)));
    v0 = v0 > 0.f ? fmaf(-z0, q.x, v0) : v0 * q.x;     // (NaN stays)
    v1 = v1 > 0.f ? fmaf(-z1, q.y, v1) : v1 * q.y;
}
__device__ __forceinline__ float gelu(float v) {
    float other = 0.f;
    gelu2(v, other);
    return v;
}

}  // namespace moe
