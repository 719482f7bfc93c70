// activation.cuh -- the activations of a linear layer and their derivatives, in
// fp32.
//
// Both are written so that infinities give the limits: the argument is kept
// finite, where the function has long reached its limit (a comparison that a
// NaN fails leaves it a NaN).  Exponentials and quotients are the hardware's
// approximations, off by some 2^-21 of the result, which a 16-bit output does
// not show.
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/linear.h"

namespace ssp {

__device__ __forceinline__ float between(float z, float lo, float hi) { return z < lo ? lo : (z > hi ? hi : z); }

__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kGeluTanh = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

// z (1 + tanh u) / 2 = z logistic(2u).
template <int ACT>
__device__ __forceinline__ float activation(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == LINEAR_ACT_GELU) {
        const float f = z < -1e30f ? -1e30f : z;
        return f * normcdff(f);
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float f = z < -1e10f ? -1e10f : z;
        return __fdividef(f, 1.0f + __expf(-2.0f * kGeluTanh * (f + kGeluCube * f * f * f)));
    }
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const float f = z < -1e30f ? -1e30f : z;
        return __fdividef(f, 1.0f + __expf(-f));
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float derivative(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
    if constexpr (ACT == LINEAR_ACT_GELU) {
        const float f = between(z, -30.0f, 30.0f);
        return normcdff(f) + f * 0.39894228040143268f * __expf(-0.5f * f * f);
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float f = between(z, -30.0f, 30.0f);
        const float p = logistic(2.0f * kGeluTanh * (f + kGeluCube * f * f * f));
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
