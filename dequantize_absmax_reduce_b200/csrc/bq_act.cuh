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

__device__ __forceinline__ float logistic(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));   // exp(-x) = 2^(-x log2 e)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

constexpr float kGeluA = 0.7978845608028654f;        // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == BQ_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    else if constexpr (ACT == BQ_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.7071067811865476f));
    else if constexpr (ACT == BQ_ACT_GELU_TANH) return z * logistic(2.0f * kGeluA * fmaf(kGeluB * z * z, z, z));
    else if constexpr (ACT == BQ_ACT_SILU) return z * logistic(z);
    else return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == BQ_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    else if constexpr (ACT == BQ_ACT_GELU)
        return fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.7071067811865476f)));
    else if constexpr (ACT == BQ_ACT_GELU_TANH) {
        const float s = logistic(2.0f * kGeluA * fmaf(kGeluB * z * z, z, z));
        // d/dz z s(2a): s + z s (1 - s) 2a'; s (1 - s) is 0 where z is so large that z a' overflows.
        const float t = s * (1.0f - s);
        return t == 0.0f ? s : fmaf(2.0f * kGeluA * z * t, fmaf(3.0f * kGeluB * z, z, 1.0f), s);
    } else if constexpr (ACT == BQ_ACT_SILU) {
        const float s = logistic(z);
        const float t = s * (1.0f - s);
        return t == 0.0f ? s : fmaf(z, t, s);
    } else return 1.0f;
}

}  // namespace bq
