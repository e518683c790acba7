// Activations of the products' epilogues and their slopes, in f32.
//
// The logistic function carries three of them: silu(z) = z s(z), and the tanh
// form of gelu is z s(2a) with a = sqrt(2/pi) (z + 0.044715 z^3), because
// (1 + tanh a) / 2 = s(2a): one exponential and one reciprocal where a tanh
// would cost several times that. s is taken as 1 / (1 + exp(-x)) with the
// hardware's exponential and reciprocal: a relative error of about 2^-21 near
// zero, growing with |x| where s itself vanishes, far below half a step of a
// 16-bit result.
#pragma once

#include "bq.h"
#include "bq_device.cuh"

namespace bq {

constexpr float kLog2e = 1.4426950408889634f;
// 1 / (1 + 2^t)
__device__ __forceinline__ float logistic_of(float t) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
__device__ __forceinline__ float logistic(float x) { return logistic_of(x * -kLog2e); }

constexpr float kGeluA = 0.7978845608028654f;        // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
// s(2a) of the tanh form: the argument is z times an even polynomial.
__device__ __forceinline__ float gelu_gate(float z) {
    return logistic_of(z * fmaf(z * z, -2.0f * kLog2e * kGeluA * kGeluB, -2.0f * kLog2e * kGeluA));
}
// z within [-lim, lim]; a NaN stays one. The slopes below are 0 or 1 to the last
// bit beyond their limits, where 0 * infinity would stand in their formulas.
__device__ __forceinline__ float clamp_nan(float z, float lim) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(lim));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-lim));
    return r;
}

// The normal distribution's tail for gelu, Phi(-x) at x >= 0, relative to its own
// size: 1 + erf leaves nothing of gelu below -5.6. Phi(-x) exp(x^2 / 2) falls
// smoothly from 1/2 to 1 / (x sqrt(2 pi)): it is taken as t times a polynomial of t =
// 1 / (1 + 0.305 x) whose eight coefficients give the least greatest relative error
// on [0, 13.5], 1e-7 (a linear program over Chebyshev points); with f32's roundings
// and the reciprocal's 10 * 2^-24. e = exp(-x^2 / 2), with which it vanishes past
// 13.2, serves the slope's density too. (Gradient of 4096 x 11008 bf16: 53 us, 75 with
// erff, 102 with erfcf; 4096 x 18432 x 7168 with bias and kept value: 620, 640, 780.)
__device__ __forceinline__ float normal_tail(float x, float& e) {
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(x, 0.305f, 1.0f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * x * (-0.5f * kLog2e)));
    float r = fmaf(0.0366991833f, t, -0.152988344f);
    r = fmaf(r, t, 0.185717046f);
    r = fmaf(r, t, -0.0379770696f);
    r = fmaf(r, t, 0.121021859f);
    r = fmaf(r, t, 0.103420801f);
    r = fmaf(r, t, 0.122466832f);
    r = fmaf(r, t, 0.121639736f);
    return r * t * e;
}
// |z|, 16 beyond it (the tail is 0 there, but not times infinity); a NaN stays one.
__device__ __forceinline__ float tail_arg(float z) {
    float x;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(fabsf(z)), "f"(16.0f));
    return x;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == BQ_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    else if constexpr (ACT == BQ_ACT_GELU) {                         // max(z, 0) - |z| Phi(-|z|)
        const float x = tail_arg(z);
        float e;
        return fmaf(-x, normal_tail(x, e), fmaxf(z, 0.0f));
    } else if constexpr (ACT == BQ_ACT_GELU_TANH) return z * gelu_gate(z);
    else if constexpr (ACT == BQ_ACT_SILU) return z * logistic(z);
    else return z;
}

// With s the logistic function of the activation's argument, d/dz z s = s (1 +
// z (1 - s) times the argument's own slope).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == BQ_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    else if constexpr (ACT == BQ_ACT_GELU) {
        const float x = tail_arg(z);
        float e;
        const float q = normal_tail(x, e);
        return fmaf(copysignf(x, z) * 0.3989422804014327f, e, z > 0.0f ? 1.0f - q : q);
    } else if constexpr (ACT == BQ_ACT_GELU_TANH) {
        const float c = clamp_nan(z, 16.0f), s = gelu_gate(c);
        const float q = c * fmaf(c * c, 6.0f * kGeluA * kGeluB, 2.0f * kGeluA);
        return fmaf(s, fmaf(-s, q, q), s);
    } else if constexpr (ACT == BQ_ACT_SILU) {
        const float c = clamp_nan(z, 126.0f), s = logistic(c);
        return fmaf(s, fmaf(-s, c, c), s);
    } else return 1.0f;
}

}  // namespace bq
