// activation.cuh -- the activations of a linear layer and their derivatives, in
// fp32.
//
// Both are written so that infinities give the limits: the argument is kept
// finite, where the function has long reached its limit (a comparison that a
// NaN fails leaves it a NaN).  Exponentials and reciprocals are single
// instructions (approximate, subnormals flushed), off by some 2^-22 of the result,
// which a 16-bit output does not show; the compiler's own forms of them spend more
// instructions on subnormals than on the rest.
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/linear.h"

namespace ssp {

__device__ __forceinline__ float between(float z, float lo, float hi) { return z < lo ? lo : (z > hi ? hi : z); }

__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-v)).
__device__ __forceinline__ float logistic(float v) { return reciprocal_fast(1.0f + exp2_fast(-kLog2e * v)); }

constexpr float kGeluTanh = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

// The normal distribution function as Phi(-x) = exp(-x^2 / 2) P(t) for x >= 0, t =
// 1 / (1 + 0.36 x): the form of Hastings' approximations (Abramowitz and Stegun
// 7.1.26), with P fitted to the least largest relative error over 0 <= x <= 14,
// 9e-7, so that the tail keeps its digits too.  Also gives exp(-z^2 / 2).  Against
// CUDA's normcdff: 2048^3 with gelu and z kept 17.9 us for 29.9.
__device__ __forceinline__ float normal_share(float z, float& bell) {
    const float t = reciprocal_fast(fmaf(0.36f, fabsf(z), 1.0f));
    bell = exp2_fast((-0.5f * kLog2e) * z * z);
    float p = fmaf(t, 0.0470564048f, -0.179765101f);
    p = fmaf(t, p, 0.180954551f);
    p = fmaf(t, p, 0.0265489823f);
    p = fmaf(t, p, 0.139719377f);
    p = fmaf(t, p, 0.141772435f);
    p = fmaf(t, p, 0.143713047f);
    p *= t * bell;
    return z > 0.0f ? 1.0f - p : p;
}

// z (1 + tanh u) / 2 = z logistic(2u).
template <int ACT>
__device__ __forceinline__ float activation(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == LINEAR_ACT_GELU) {
        const float f = z < -1e10f ? -1e10f : z;
        float bell;
        return f * normal_share(f, bell);
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float f = z < -1e10f ? -1e10f : z;
        return f * logistic(2.0f * kGeluTanh * fmaf(kGeluCube * f * f, f, f));
    }
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const float f = z < -1e30f ? -1e30f : z;
        return f * logistic(f);
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float derivative(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
    if constexpr (ACT == LINEAR_ACT_GELU) {
        const float f = between(z, -30.0f, 30.0f);
        float bell;
        const float share = normal_share(f, bell);
        return fmaf(f * 0.39894228040143268f, bell, share);
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float f = between(z, -30.0f, 30.0f);
        const float p = logistic(2.0f * kGeluTanh * fmaf(kGeluCube * f * f, f, f));
        return p + f * p * (1.0f - p) * (2.0f * kGeluTanh * (1.0f + 3.0f * kGeluCube * f * f));
    }
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const float f = between(z, -120.0f, 120.0f);
        const float p = logistic(f);
        return p + f * p * (1.0f - p);
    }
    return 1.0f;
}

// f(the activation's number as a constant): one branch for a whole run of values.
template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    switch (act) {
        case LINEAR_ACT_RELU: f(std::integral_constant<int, LINEAR_ACT_RELU>{}); break;
        case LINEAR_ACT_GELU: f(std::integral_constant<int, LINEAR_ACT_GELU>{}); break;
        case LINEAR_ACT_GELU_TANH: f(std::integral_constant<int, LINEAR_ACT_GELU_TANH>{}); break;
        case LINEAR_ACT_SILU: f(std::integral_constant<int, LINEAR_ACT_SILU>{}); break;
        default: break;
    }
}

}  // namespace ssp
