// ortho.cuh -- what orthogonalize's two ways share: the gradient's elements, the
// sum of their squares, and the scales of the fp16 tensors.
#pragma once
#include <cmath>

#include "product.cuh"

namespace ssp {

struct OrthoInput {
    const void* g = nullptr;
    long long ld = 0, stride = 0;
};

// Eight elements of matrix b's row from column c on, as they lie, zeros past the
// `left` that are wanted.
struct Raw {
    uint4 lo, hi;  // hi: fp32 alone
};
template <int TYPE>
__device__ __forceinline__ Raw load_raw(const OrthoInput& in, int b, int row, int c, int left) {
    const long long i = static_cast<long long>(b) * in.stride + static_cast<long long>(row) * in.ld + c;
    Raw r = {};
    if constexpr (TYPE == QUANT_F32) {
        const uint32_t* s = static_cast<const uint32_t*>(in.g) + i;
        if (left >= 8) {
            r.lo = reinterpret_cast<const uint4*>(s)[0];
            r.hi = reinterpret_cast<const uint4*>(s)[1];
        } else {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = e < left ? s[e] : 0u;
            r = {make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7])};
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(in.g) + i;
        if (left >= 8) {
            r.lo = *reinterpret_cast<const uint4*>(s);
        } else {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = e < left ? s[e] : 0u;
            r.lo = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
        }
    }
    return r;
}
template <int TYPE>
__device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
    const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    if constexpr (TYPE == QUANT_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16<TYPE == QUANT_BF16>(w[e]);
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// A thread's sum of squares.  Sums of squares of elements beyond 2^45 or below
// 2^-45 may leave fp32's range: a group of eight whose largest is such is scaled by
// 2^-80 or 2^90 and summed apart.  (Beside a larger element of its group, a square
// that underflows is too small to count.)
struct SquareSum {
    float sum = 0.0f, large = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(const float (&v)[8]) {
        float most = 0.0f, s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            most = fmaxf(most, fabsf(v[e]));
            s = fmaf(v[e], v[e], s);
        }
        if (most <= 0x1p45f && (most >= 0x1p-45f || most == 0.0f)) {
            sum += s;  // a NaN among the eight is in s
        } else {
            const float by = most > 1.0f ? 0x1p-80f : 0x1p90f;
            s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[e] * by, v[e] * by, s);
            if (most > 1.0f) large += s;
            else small += s;
        }
    }
    // The warp's, for lane 0.  (64-bit arithmetic is slow here: one thread a warp.)
    __device__ __forceinline__ double warp_total() {
        sum = warp_sum(sum);
        large = warp_sum(large);
        small = warp_sum(small);
        if ((threadIdx.x & 31) != 0) return 0.0;
        return static_cast<double>(sum) + static_cast<double>(large) * 0x1p160 + static_cast<double>(small) * 0x1p-180;
    }
};

// The first X is G 2^e with a norm between 2^exponent and twice that, and t = 2^-e /
// (|G| + eps) is what is left of the norm: 2^e in two factors, since it may lie
// beyond fp32's exponents, and t.  t is NaN where the norm is not finite; where it
// is 0, X is zeros, or with eps = 0 NaN.
__device__ __forceinline__ void first_factors(double squares, int exponent, float eps, float* f) {
    const double norm = sqrt(squares);
    int e = 0;
    if (norm > 0.0 && norm < 1e300) e = exponent - ilogb(norm);
    float t = nanf("");
    if (norm < 1e300)
        t = norm == 0.0 && eps > 0.0f ? 1.0f : static_cast<float>(ldexp(1.0, -e) / (norm + static_cast<double>(eps)));
    f[0] = ldexpf(1.0f, e / 2);
    f[1] = ldexpf(1.0f, e - e / 2);
    f[2] = t;
}

// ---------------------------------------------------------------- host side
// Powers of two: of A and b A + c A^2 (which have singular values below 4), of X
// between the steps, and the first X's norm, whose largest element is below 2^15.
struct OrthoScales {
    float a, x;
    int exponent;
};
inline OrthoScales ortho_scales(int64_t rows, int64_t cols) {
    const int64_t n = rows < cols ? rows : cols, m = rows < cols ? cols : rows;
    const int la = std::ilogb(static_cast<double>(n));
    const int e = std::ilogb(std::sqrt(static_cast<double>(rows) * static_cast<double>(cols)));
    return {std::ldexp(1.0f, la < 14 ? la : 14), std::ldexp(1.0f, std::ilogb(std::sqrt(static_cast<double>(m)))),
            e < 14 ? e : 14};
}

}  // namespace ssp
