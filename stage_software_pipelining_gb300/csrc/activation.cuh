// activation.cuh -- the activations of a linear layer and their derivatives, in
// fp32, two values at a time.
//
// An epilogue has about as many instruction slots for a value as its product has
// for K = 30, so these are written to the count: sums and products on packed pairs
// (f32x2, two results an instruction), one reciprocal for two denominators (1/a =
// b/(ab)), exponentials and reciprocals as single instructions (approximate,
// subnormals flushed: the compiler's own forms spend more on subnormals than on the
// rest).  2048^3 with gelu and z kept: 29.9 us with CUDA's normcdff, 22.5 with the
// approximation below one value at a time.
//
// Errors, of these steps emulated in fp32 (with exact exp2 and reciprocals) for all
// fp16 z from -12 to 12 (gelu_tanh from -7.5): of an activation 2^-19 of its value and
// of a derivative 2^-19 of its largest, some 1; below -4, where both are small, 2^-17 of
// their own values, because the exponent is itself rounded.  A 16-bit output shows none
// of them.  Arguments are limited to where the function has reached its limit to within
// 3e-17 (so that the product of two denominators stays finite); with that, infinities
// give the limits; a NaN stays in its own value.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/linear.h"

namespace ssp {

// Two fp32 values in one register pair.
using Pair = uint64_t;

__device__ __forceinline__ Pair make_pair2(float x, float y) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 both(Pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ Pair pair_of(float v) { return make_pair2(v, v); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ float at_least(float v, float lo) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lo));
    return r;
}
__device__ __forceinline__ float at_most(float v, float hi) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(hi));
    return r;
}
__device__ __forceinline__ Pair at_least(Pair p, float lo) {
    const float2 v = both(p);
    return make_pair2(at_least(v.x, lo), at_least(v.y, lo));
}
__device__ __forceinline__ Pair within(Pair p, float limit) {
    const float2 v = both(p);
    return make_pair2(at_most(at_least(v.x, -limit), limit), at_most(at_least(v.y, -limit), limit));
}

// At least lo, and lo for a NaN: what goes into a shared reciprocal must not take
// one value's NaN to the other.  (It comes back by the factor beside it.)
__device__ __forceinline__ Pair finite_from(Pair p, float lo) {
    const float2 v = both(p);
    return make_pair2(fmaxf(v.x, lo), fmaxf(v.y, lo));
}

__device__ __forceinline__ Pair exp2_of(Pair p) {
    float2 v = both(p);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.y));
    return make_pair2(v.x, v.y);
}

// 1/a and 1/b of the pair (a, b), whose product is finite and normal.
__device__ __forceinline__ Pair reciprocals(Pair p) {
    const float2 v = both(p);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v.x * v.y));
    return mul2(make_pair2(v.y, v.x), pair_of(r));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluTanh = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
constexpr float kBellTop = 0.39894228040143268f;   // 1 / sqrt(2 pi)
// exp(43) = 2^62: the product of two such is finite.
constexpr float kLogisticEnd = 43.0f;
constexpr float kGeluTanhEnd = 7.6f;  // where gelu_tanh's logistic has that argument

// 1 / (1 + exp(-v)) for v from -kLogisticEnd to infinity; that of -kLogisticEnd
// below it and for a NaN.
__device__ __forceinline__ Pair logistic(Pair v) {
    const Pair e = exp2_of(mul2(finite_from(v, -kLogisticEnd), pair_of(-kLog2e)));
    return reciprocals(add2(e, pair_of(1.0f)));
}

// The argument of gelu_tanh's logistic: (1 + tanh u) / 2 = logistic(2u).
__device__ __forceinline__ Pair gelu_tanh_argument(Pair z) {
    return mul2(z, fma2(mul2(z, z), pair_of(2.0f * kGeluTanh * kGeluCube), pair_of(2.0f * kGeluTanh)));
}

// -Phi(-|z|) = -exp(-z^2 / 2) P(t), t = 1 / (1 + 0.36 |z|), and exp(-z^2 / 2): the
// form of Hastings' approximations (Abramowitz and Stegun 7.1.26), with P fitted to
// the least largest relative error over 0 <= |z| <= 14, 9e-7, so that the tail keeps
// its digits too.  `size` is |z|, limited.
__device__ __forceinline__ Pair normal_tail(Pair z, Pair size, Pair& bell) {
    const Pair t = reciprocals(fma2(size, pair_of(0.36f), pair_of(1.0f)));
    bell = exp2_of(mul2(mul2(z, z), pair_of(-0.5f * kLog2e)));
    Pair p = fma2(t, pair_of(-0.0470564048f), pair_of(0.179765101f));
    p = fma2(t, p, pair_of(-0.180954551f));
    p = fma2(t, p, pair_of(-0.0265489823f));
    p = fma2(t, p, pair_of(-0.139719377f));
    p = fma2(t, p, pair_of(-0.141772435f));
    p = fma2(t, p, pair_of(-0.143713047f));
    return mul2(mul2(p, t), bell);
}
__device__ __forceinline__ Pair size_of(Pair z) {
    const float2 v = both(z);
    return make_pair2(fminf(fabsf(v.x), 100.0f), fminf(fabsf(v.y), 100.0f));
}

// 1 for v >= 0, else 0.
__device__ __forceinline__ float step_of(float v) {
    float r;
    asm("set.ge.f32.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

template <int ACT>
__device__ __forceinline__ Pair activation(Pair z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return at_least(z, 0.0f);
    if constexpr (ACT == LINEAR_ACT_GELU) {
        // max(z, 0) - |z| Phi(-|z|); a NaN comes through the tail.
        Pair bell;
        const Pair size = size_of(z), tail = normal_tail(z, size, bell);
        const float2 v = both(z);
        return fma2(size, tail, make_pair2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const Pair f = at_least(z, -kGeluTanhEnd);
        return mul2(f, logistic(gelu_tanh_argument(f)));
    }
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const Pair f = at_least(z, -kLogisticEnd);
        return mul2(f, logistic(f));
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ Pair derivative(Pair z) {
    if constexpr (ACT == LINEAR_ACT_RELU) {
        const float2 v = both(z);
        return make_pair2(v.x <= 0.0f ? 0.0f : 1.0f, v.y <= 0.0f ? 0.0f : 1.0f);
    }
    if constexpr (ACT == LINEAR_ACT_GELU) {
        // Phi(z) + z phi(z) = step + (2 step - 1) w, step 0 below zero and else 1, w =
        // |z| phi(z) - Phi(-|z|): below zero nothing is added to w, which keeps its
        // digits.  A NaN comes through the bell.  (8192^2 act_grad 80.1 us and 4096^2
        // linear_dx of sums of 64 25.3; with signs by copysign 81.1 and 25.8.)
        const float2 v = both(z);
        const Pair size = make_pair2(fminf(fabsf(v.x), 30.0f), fminf(fabsf(v.y), 30.0f));
        const Pair step = make_pair2(step_of(v.x), step_of(v.y));
        Pair bell;
        const Pair tail = normal_tail(z, size, bell);
        const Pair w = fma2(mul2(size, pair_of(kBellTop)), bell, tail);
        return fma2(fma2(step, pair_of(2.0f), pair_of(-1.0f)), w, step);
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const Pair f = within(z, kGeluTanhEnd);
        const Pair p = logistic(gelu_tanh_argument(f));
        const Pair k = fma2(mul2(f, f), pair_of(6.0f * kGeluTanh * kGeluCube), pair_of(2.0f * kGeluTanh));
        const Pair rest = fma2(p, pair_of(-1.0f), pair_of(1.0f));
        return mul2(p, fma2(mul2(f, k), rest, pair_of(1.0f)));
    }
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const Pair f = within(z, kLogisticEnd);
        const Pair p = logistic(f);
        return mul2(p, fma2(f, fma2(p, pair_of(-1.0f), pair_of(1.0f)), pair_of(1.0f)));
    }
    return pair_of(1.0f);
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
