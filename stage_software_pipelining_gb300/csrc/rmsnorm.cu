// rmsnorm.cu -- the residual's addition, the root-mean-square norm and the
// 8-bit rows with a scale each, in one kernel:
//
//     h = x + residual,  y = h / sqrt(mean(h^2) + eps) * w,
//     scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
//
// A row is read once and stays in registers as fp32.  y's largest magnitude is
// rstd * max|h w|, so the sum of squares and the maximum come from one pass and
// one reduction, after which every output is written.  Nothing is rounded
// between the input and an output.
//
// Bound by memory: per element two reads and, for the 8-bit form, a write of
// the sum and of one byte.  Rows of up to 1024 elements (16-bit) take a warp
// each, longer ones a block (row_kernel); a row off 16-byte boundaries, or too long
// for a block's registers, goes by way of shared memory (staged_kernel), and one
// that does not fit there either is read twice (wide_kernel).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <mutex>
#include <type_traits>

#include "../../include/quant.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant.h"

namespace ssp {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: 1/scale stays finite

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// The larger of two values, NaN if either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// VEC adjacent elements of a row as they lie in memory: 16 bytes, or one
// element where rows do not start on 16-byte boundaries.
template <typename T, int VEC>
struct Pack {
    uint4 u;
    __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
    // Every element the same.
    __device__ __forceinline__ void fill(float v) {
        T e[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(v);
        u.x = u.y = u.z = u.w = *reinterpret_cast<const uint32_t*>(e);
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            } else {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <typename T>
struct Pack<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T* p) { u = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = u; }
    __device__ __forceinline__ void fill(float v) { u = from_f32<T>(v); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(u); }
    __device__ __forceinline__ void set(const float (&f)[1]) { u = from_f32<T>(f[0]); }
};

struct Stats {
    float ss;  // sum of h^2
    float am;  // max |h w|, or max |h| without a norm
};

__device__ __forceinline__ Stats warp_join(Stats s) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        s.ss += __shfl_xor_sync(0xffffffffu, s.ss, o);
        s.am = max_nan(s.am, __shfl_xor_sync(0xffffffffu, s.am, o));
    }
    return s;
}

// The block's Stats in every thread, in the same order every time.
__device__ __forceinline__ Stats block_join(Stats s, Stats* buf) {
    s = warp_join(s);
    const int lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x >> 5);
    if (lane == 0) buf[threadIdx.x >> 5] = s;
    __syncthreads();
    // The warps' Stats once in every run of `run` lanes (warps rounded up to a
    // power of two), joined within the run.
    const int run = 1 << (32 - __clz(warps - 1));
    const int w = lane & (run - 1);
    s = w < warps ? buf[w] : Stats{0.0f, 0.0f};
    for (int o = 1; o < run; o *= 2) {
        s.ss += __shfl_xor_sync(0xffffffffu, s.ss, o);
        s.am = max_nan(s.am, __shfl_xor_sync(0xffffffffu, s.am, o));
    }
    return s;
}

// rstd, scale and 1/scale of a row from its Stats.  A row whose largest y is not
// finite has neither a scale nor 8-bit values: both are NaN, also where the
// formula would give an infinite scale and zeros.  (A scale that is a number lies
// in [2^-126, 2^120], so 1/scale is one too.)
//
// Quotients often lie half-way between two e4m3 values where the scale has few
// bits (largest 21 of small integers: 57/64 over 3/64 is 19) and must not be off
// by an ulp there.  So the scale, max / 448, is correctly rounded (what the product
// with the rounded reciprocal leaves of the dividend is exact, and its share closes
// the gap: Markstein's division), and 1/scale is held in two parts, 2^-46 off at
// most: y inv + y rest is then rounded once, and exact where the quotient is.  The
// second part is positive, so that both products of a -0 are one.
struct Factors {
    float rstd, scale, inv, rest;
};
__device__ __forceinline__ Factors row_factors(const NormLaunch& p, Stats s, float eps) {
    Factors f;
    f.rstd = p.weight ? rsqrtf(fmaf(s.ss, p.inv_cols, eps)) : 1.0f;
    const float most = f.rstd * s.am;
    constexpr float kInv = 1.0f / kE4m3Max;
    const float v = most * kInv;
    f.scale = most <= FLT_MAX ? fmaxf(fmaf(fmaf(-v, kE4m3Max, most), kInv, v), kScaleMin) : __int_as_float(0x7fffffff);
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(f.scale));  // within an ulp
    f.inv = __int_as_float(__float_as_int(r) - 1);            // and below 1/scale
    f.rest = fmaf(-f.scale, f.inv, 1.0f) * f.inv;
    return f;
}

// Two products or multiply-adds in one instruction, rounded as two.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// y = h rstd g.
template <int VEC>
__device__ __forceinline__ void normed(const float (&h)[VEC], const float (&g)[VEC], const Factors& f, float (&y)[VEC]) {
    if constexpr (VEC == 1) {
        y[0] = h[0] * f.rstd * g[0];
    } else {
        const uint64_t rstd = two(f.rstd, f.rstd);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const uint64_t v = mul2(mul2(two(h[e], h[e + 1]), rstd), two(g[e], g[e + 1]));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(y[e]), "=f"(y[e + 1]) : "l"(v));
        }
    }
}

// e4m3(y / scale).
template <int VEC>
__device__ __forceinline__ void store_q(uint8_t* q, const float (&y)[VEC], const Factors& f) {
    if constexpr (VEC == 1) {
        *q = __nv_cvt_float_to_fp8(fmaf(y[0], f.inv, y[0] * f.rest), __NV_SATFINITE, __NV_E4M3);
    } else {
        const uint64_t inv = two(f.inv, f.inv), rest = two(f.rest, f.rest);
        alignas(VEC) uint16_t v[VEC / 2];
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const uint64_t yy = two(y[e], y[e + 1]), r = fma2(yy, inv, mul2(yy, rest));
            float2 o;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
            v[e / 2] = __nv_cvt_float2_to_fp8x2(o, __NV_SATFINITE, __NV_E4M3);
        }
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(v);
        else *reinterpret_cast<uint32_t*>(q) = *reinterpret_cast<const uint32_t*>(v);
    }
}

// Whether a row's Stats have left fp32's range although its y need not: the
// squares of |h| above 1.8e19 / sqrt(cols) sum to infinity, those below 2^-63 lose
// their last bits (eps not covering them), and h w may do either before rstd
// brings it back.  Such a row's Stats are taken again from h f with f = 2^-n near
// 1 / max(max|h|, sqrt(eps)): y = h f / sqrt(mean((h f)^2) + eps f^2) * w, every
// product by f exact.  (Rows of zeros keep their Stats; without a weight only
// max|h| counts, which is exact.)
__device__ __forceinline__ bool out_of_range(const NormLaunch& p, Stats s) {
    // Two comparisons settle ordinary rows (2^-100 to FLT_MAX, as integers).
    auto ordinary = [](float v) { return __float_as_uint(v) - 0x0d800000u <= 0x7f7fffffu - 0x0d800000u; };
    if (!p.weight || (ordinary(fmaf(s.ss, p.inv_cols, p.eps)) && ordinary(s.am))) return false;
    const float v = fmaf(s.ss, p.inv_cols, p.eps);
    if (!(v >= 0x1p-100f && v <= FLT_MAX)) return true;
    return p.scale && (!(s.am <= FLT_MAX) || (s.am < 0x1p-100f && s.ss > 0.0f));
}
// f, 1 for what is not finite; m = max|h|.
__device__ __forceinline__ float range_factor(float m, float eps) {
    const float t = max_nan(m, sqrtf(eps));
    const int e = min(max(__float_as_int(t) >> 23, 1), 253);
    return t <= FLT_MAX ? __int_as_float((254 - e) << 23) : 1.0f;
}

// h of element i of a row; without a residual x itself, the sign of a zero included.
template <typename T>
struct RowIn {
    const T *x, *r, *w;
    __device__ __forceinline__ RowIn(const NormLaunch& p, long long row)
        : x(static_cast<const T*>(p.x) + row * p.ldx),
          r(p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr),
          w(static_cast<const T*>(p.weight)) {}
    __device__ __forceinline__ float h(int i) const { return r ? to_f32(x[i]) + to_f32(r[i]) : to_f32(x[i]); }
};

// The Stats of a row out of range, read again by its threads, of which this is
// the t-th: f, with s and eps as row_factors wants them for h f.
template <typename T, bool WARP>
__device__ __forceinline__ float scaled_stats(const NormLaunch& p, long long row, int t, int threads, Stats* buf,
                                              Stats& s, float& eps) {
    const RowIn<T> in(p, row);
    const int n = static_cast<int>(p.cols);
    auto join = [&](Stats v) {
        if (WARP) return warp_join(v);
        __syncthreads();  // buf has been read
        return block_join(v, buf);
    };
    float m = 0.0f;
#pragma unroll 1
    for (int i = t; i < n; i += threads) m = max_nan(m, fabsf(in.h(i)));
    const float f = range_factor(join({0.0f, m}).am, eps);
    eps = eps * f * f;
    s = {0.0f, 0.0f};
#pragma unroll 1
    for (int i = t; i < n; i += threads) {
        const float h = in.h(i) * f;
        s.ss = fmaf(h, h, s.ss);
        s.am = max_nan(s.am, fabsf(h * to_f32(in.w[i])));
    }
    s = join(s);
    return f;
}

// A row's outputs, read again; `by` scales h as the Factors expect.  Every element
// is read and written by the same thread, so outputs may lie over inputs.
template <typename T>
__device__ __forceinline__ void write_row(const NormLaunch& p, long long row, int t, int threads, const Factors& f,
                                          float by) {
    const RowIn<T> in(p, row);
    const int n = static_cast<int>(p.cols);
    if (p.scale && t == 0) p.scale[row] = f.scale;
#pragma unroll 1
    for (int i = t; i < n; i += threads) {
        const float h = in.h(i);
        const float y = in.w ? h * by * f.rstd * to_f32(in.w[i]) : h;
        if (p.residual_out) static_cast<T*>(p.residual_out)[row * p.ldro + i] = from_f32<T>(h);
        if (p.y) static_cast<T*>(p.y)[row * p.ldy + i] = from_f32<T>(y);
        const float one[1] = {y};
        if (p.q) store_q<1>(static_cast<uint8_t*>(p.q) + row * p.ldq + i, one, f);
    }
}

// A row in registers: thread t of the row's `threads` holds packs t, t +
// threads, ..., NCH of them.  WARP: a warp a row, blockDim/32 rows a block;
// otherwise a block a row.
// Threads a block may have: what its registers leave room for (x, residual,
// weight and h of VEC * NCH elements a thread).
constexpr int max_threads(int size, int vec, int nch) { return (vec == 1 ? 4 : size) * vec * nch <= 32 ? 1024 : 512; }

template <typename T, int VEC, int NCH, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : max_threads(sizeof(T), VEC, NCH)) row_kernel(const NormLaunch p) {
    using P = Pack<T, VEC>;
    __shared__ Stats buf[WARP ? 1 : 32];
    griddep_launch_dependents();
    griddep_wait();
    const int threads = WARP ? 32 : static_cast<int>(blockDim.x);
    const int t = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const long long row = WARP ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                               : static_cast<long long>(blockIdx.x);
    if (WARP && row >= p.rows) return;
    const int packs = static_cast<int>(p.cols) / VEC;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
    const T* w = static_cast<const T*>(p.weight);
    // Every load is on its way before the first value is used.  Absent inputs
    // are neutral ones: a residual of -0 (x + -0 is x, signs of zero included)
    // and weights of 1.
    P xv[NCH], rv[NCH], wv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
        if (t + c * threads < packs) xv[c].load(x + (t + c * threads) * VEC);
    if (p.residual) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            if (t + c * threads < packs) rv[c].load(r + (t + c * threads) * VEC);
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) rv[c].fill(-0.0f);
    }
    if (p.weight) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            if (t + c * threads < packs) wv[c].load(w + (t + c * threads) * VEC);
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) wv[c].fill(1.0f);
    }
    float h[NCH][VEC];
    Stats s = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        if (t + c * threads < packs) {
            float a[VEC], b[VEC], g[VEC];
            xv[c].get(a);
            rv[c].get(b);
            wv[c].get(g);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                if constexpr (VEC == 1) {
                    const float v = a[e] + b[e];
                    h[c][e] = v;
                    s.ss = fmaf(v, v, s.ss);
                    s.am = max_nan(s.am, fabsf(v * g[e]));
                } else {
                    const uint64_t v = add2(two(a[e], a[e + 1]), two(b[e], b[e + 1]));
                    const uint64_t u = mul2(v, two(g[e], g[e + 1]));
                    float2 o;
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(h[c][e]), "=f"(h[c][e + 1]) : "l"(v));
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(u));
                    s.ss = fmaf(h[c][e], h[c][e], s.ss);
                    s.ss = fmaf(h[c][e + 1], h[c][e + 1], s.ss);
                    s.am = max_nan(s.am, fabsf(o.x));
                    s.am = max_nan(s.am, fabsf(o.y));
                }
            }
        }
    }
    s = WARP ? warp_join(s) : block_join(s, buf);
    T* ro = static_cast<T*>(p.residual_out) + row * p.ldro;
    // Nothing is written yet: such a row is read again, which leaves the others'
    // registers as they are (h kept through the branch cost 5 to 13 % on short rows).
    if (out_of_range(p, s)) {
        float eps = p.eps;
        const float by = scaled_stats<T, WARP>(p, row, t, threads, buf, s, eps);
        write_row<T>(p, row, t, threads, row_factors(p, s, eps), by);
        return;
    }
    const Factors f = row_factors(p, s, p.eps);
    if (p.scale && t == 0) p.scale[row] = f.scale;
    T* yo = static_cast<T*>(p.y) + row * p.ldy;
    uint8_t* q = static_cast<uint8_t*>(p.q) + row * p.ldq;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int i = (t + c * threads) * VEC;
        if (t + c * threads < packs) {
            P o;
            if (p.residual_out) {
                o.set(h[c]);
                o.store(ro + i);
            }
            float g[VEC], y[VEC];
            wv[c].get(g);
            normed(h[c], g, f, y);
            if (p.y) {
                o.set(y);
                o.store(yo + i);
            }
            if (p.q) store_q<VEC>(q + i, y, f);
        }
    }
}

// Rows that do not start on 16-byte boundaries (an odd width), or too long for
// a block's registers: the row lies in shared memory as fp32 on the way.  x, the
// residual and its sum are moved 16 bytes at a time from the first boundary in
// the row on, where they agree on it (SAME), the weights, q and an aligned y
// from the row's first element on; shared memory turns one into the other.
// Each element of an input is read before any thread writes an output over it.
struct Staged {
    int same;   // x, residual, residual_out start alike within 16 bytes, row by row
    int y_same; // y too
    int w_vec, q_vec, y_vec;  // on 16-byte (q: VEC-byte) boundaries
};

template <typename T>
__global__ void __launch_bounds__(512) staged_kernel(const NormLaunch p, const Staged st) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ float hb[];
    __shared__ Stats buf[32];
    griddep_launch_dependents();
    griddep_wait();
    const long long row = blockIdx.x;
    const int n = static_cast<int>(p.cols), t = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const T* w = static_cast<const T*>(p.weight);
    T* ro = p.residual_out ? static_cast<T*>(p.residual_out) + row * p.ldro : nullptr;
    T* yo = p.y ? static_cast<T*>(p.y) + row * p.ldy : nullptr;
    uint8_t* q = p.q ? static_cast<uint8_t*>(p.q) + row * p.ldq : nullptr;
    auto at = [](int i) { return i + (i >> 3); };  // no bank conflicts for runs of VEC a lane
    // Whole packs lie in [head, tail).
    int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / sizeof(T));
    if (head > n || !st.same) head = n;
    const int packs = (n - head) / VEC, tail = head + packs * VEC;
    float ss = 0.0f;
    auto take = [&](int i) {
        float h = to_f32(x[i]);
        if (r) h += to_f32(r[i]);
        ss = fmaf(h, h, ss);
        hb[at(i)] = h;
        if (ro) ro[i] = from_f32<T>(h);
    };
    constexpr int U = 2;  // packs on their way at a time
    for (int j = t; j < packs; j += U * nt) {
        Pack<T, VEC> xv[U], rv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = head + (j + u * nt) * VEC;
            if (j + u * nt < packs) {
                xv[u].load(x + i);
                if (r) rv[u].load(r + i);
                else rv[u].fill(-0.0f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = head + (j + u * nt) * VEC;
            if (j + u * nt < packs) {
                float a[VEC], b[VEC];
                xv[u].get(a);
                rv[u].get(b);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    a[e] += b[e];
                    ss = fmaf(a[e], a[e], ss);
                    hb[at(i + e)] = a[e];
                }
                if (ro) {
                    xv[u].set(a);
                    xv[u].store(ro + i);
                }
            }
        }
    }
    for (int i = t; i < head; i += nt) take(i);
    for (int i = tail + t; i < n; i += nt) take(i);
    __syncthreads();
    // h and the weights of elements [i, i + VEC), 0 past the row.
    auto both = [&](int i, float (&h)[VEC], float (&g)[VEC]) {
        const bool whole = i + VEC <= n;
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = i + e < n ? hb[at(i + e)] : 0.0f;
        Pack<T, VEC> wv;
        if (!w) {
            wv.fill(1.0f);
            wv.get(g);
        } else if (whole && st.w_vec) {
            wv.load(w + i);
            wv.get(g);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = i + e < n ? to_f32(w[i + e]) : 0.0f;
        }
    };
    float am = 0.0f;
    if (p.scale)
        for (int i = t * VEC; i < n; i += nt * VEC) {
            float h[VEC], g[VEC];
            both(i, h, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) am = max_nan(am, fabsf(h[e] * g[e]));
        }
    Stats s = block_join({ss, am}, buf);
    float eps = p.eps;
    if (out_of_range(p, s)) {
        float m = 0.0f;
#pragma unroll 1
        for (int i = t; i < n; i += nt) m = max_nan(m, fabsf(hb[at(i)]));
        __syncthreads();  // buf has been read
        const float f = range_factor(block_join({0.0f, m}, buf).am, eps);
        eps = eps * f * f;
        s = {0.0f, 0.0f};
#pragma unroll 1
        for (int i = t; i < n; i += nt) {
            const float h = hb[at(i)] * f;
            hb[at(i)] = h;
            s.ss = fmaf(h, h, s.ss);
            s.am = max_nan(s.am, fabsf(h * to_f32(w[i])));
        }
        __syncthreads();
        s = block_join(s, buf);
    }
    const Factors f = row_factors(p, s, eps);
    if (p.scale && t == 0) p.scale[row] = f.scale;
    if (!yo && !q) return;
    const bool y_turned = yo && st.y_same && !st.y_vec;  // y leaves by way of shared memory
    for (int i = t * VEC; i < n; i += nt * VEC) {
        float h[VEC], g[VEC];
        both(i, h, g);
        const bool whole = i + VEC <= n;
        normed(h, g, f, h);
        if (yo) {
            if (y_turned) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i + e < n) hb[at(i + e)] = h[e];
            } else if (whole && st.y_vec) {
                Pack<T, VEC> o;
                o.set(h);
                o.store(yo + i);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i + e < n) yo[i + e] = from_f32<T>(h[e]);
            }
        }
        if (q) {
            if (whole && st.q_vec) {
                store_q<VEC>(q + i, h, f);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float one[1] = {h[e]};
                    if (i + e < n) store_q<1>(q + i + e, one, f);
                }
            }
        }
    }
    if (!y_turned) return;
    __syncthreads();
#pragma unroll 1  // unrolled, fp16's takes 53 registers for 40: 8000 x 2541 with q 41.6 us for 38.5
    for (int j = t; j < packs; j += nt) {
        const int i = head + j * VEC;
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = hb[at(i + e)];
        Pack<T, VEC> o;
        o.set(y);
        o.store(yo + i);
    }
    for (int i = t; i < head; i += nt) yo[i] = from_f32<T>(hb[at(i)]);
    for (int i = tail + t; i < n; i += nt) yo[i] = from_f32<T>(hb[at(i)]);
}

// A row too long for shared memory as well: one pass for its Stats, one that
// reads it again and writes.
template <typename T>
__global__ void __launch_bounds__(1024) wide_kernel(const NormLaunch p) {
    __shared__ Stats buf[32];
    griddep_launch_dependents();
    griddep_wait();
    const long long row = blockIdx.x;
    const int t = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x), n = static_cast<int>(p.cols);
    const RowIn<T> in(p, row);
    Stats s = {0.0f, 0.0f};
    for (int i = t; i < n; i += threads) {
        const float h = in.h(i);
        s.ss = fmaf(h, h, s.ss);
        s.am = max_nan(s.am, fabsf(in.w ? h * to_f32(in.w[i]) : h));
    }
    s = block_join(s, buf);
    float eps = p.eps, by = 1.0f;
    if (out_of_range(p, s)) by = scaled_stats<T, false>(p, row, t, threads, buf, s, eps);
    write_row<T>(p, row, t, threads, row_factors(p, s, eps), by);
}

using Kernel = void (*)(const NormLaunch);

template <typename... Args>
int launch(void (*k)(Args...), int64_t grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess ? GEMM_OK
                                                                                              : GEMM_ERR_LAUNCH;
}

// Rows whose packs (VEC elements) are whole and aligned.  Few threads with
// several packs each hold more loads in flight for their registers than many
// with one, and their reductions cost less: 8191 x 8192 bf16 with q takes 69 us
// with 256 threads of 4 packs (the bytes at 6.87 TB/s), 77 with 512 of 2 and 85
// with 1024 of 1.  Where rows are fewer than two an SM, one row's time counts:
// one pack a thread, as many threads as that takes.  False: not for these rows.
template <typename T, int VEC>
bool launch_rows(const NormLaunch& L, cudaStream_t stream, int* status) {
    const int64_t packs = (L.cols + VEC - 1) / VEC;
    if (packs <= 128) {  // a warp a row
        Kernel k = packs <= 32   ? row_kernel<T, VEC, 1, true>
                   : packs <= 64 ? row_kernel<T, VEC, 2, true> : row_kernel<T, VEC, 4, true>;
        *status = launch(k, (L.rows + 3) / 4, 128, 0, stream, L);
        return true;
    }
    constexpr int kMost = VEC == 1 || sizeof(T) == 4 ? 8 : 4;
    const bool few = L.rows <= 2 * tc_current_device_sms();
    // One element at a time costs more instructions the longer the row, staged_kernel
    // two more passes over shared memory and their barriers.  16-bit, with q: 400 x
    // 3501 5.1 us to 6.4 of staged_kernel, 1000 x 2001 5.9 to 6.5, x 3001 9.5 to 7.8,
    // 8000 x 1201 25.0 to 23.1, x 2541 52.1 to 36.6.  fp32: 2000 x 4001 24.6 to 25.4,
    // 4000 x 2001 22.5 to 24.4, x 3001 38.3 to 34.1.
    const bool many = L.rows > 12 * tc_current_device_sms();
    const int64_t longest = sizeof(T) == 4 ? (many ? 2560 : 4096) : many ? 1280 : 2560;
    if (VEC == 1 && !few && packs > longest) return false;
    int nch = few ? (VEC == 1 ? 4 : 1) : VEC == 1 ? 8 : 4;
    while (nch <= kMost && packs > static_cast<int64_t>(max_threads(sizeof(T), VEC, nch)) * nch) nch *= 2;
    if (nch > kMost) return false;
    Kernel k = nch == 1   ? row_kernel<T, VEC, 1, false>
               : nch == 2 ? row_kernel<T, VEC, 2, false> : row_kernel<T, VEC, 4, false>;
    if constexpr (kMost >= 8)
        if (nch == 8) k = row_kernel<T, VEC, 8, false>;
    const int threads = static_cast<int>(((packs + nch - 1) / nch + 31) / 32 * 32);
    *status = launch(k, L.rows, threads, 0, stream, L);
    return true;
}

// Whether a matrix's rows all start on `to`-byte boundaries.
bool rows_on(const void* p, int64_t ld, int64_t rows, int64_t size, uintptr_t to) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0 &&
                  (rows <= 1 || (ld * size) % static_cast<int64_t>(to) == 0));
}

// Whether two matrices' rows start alike within 16 bytes.
bool alike(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t size) {
    return !b || ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) % 16 == 0 &&
                  (rows <= 1 || (lda - ldb) * size % 16 == 0));
}

template <typename T>
int launch_type(const NormLaunch& L, cudaStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int64_t S = sizeof(T);
    Staged st;
    st.w_vec = rows_on(L.weight, 0, 1, S, 16);
    st.q_vec = rows_on(L.q, L.ldq, L.rows, 1, VEC);
    st.y_vec = rows_on(L.y, L.ldy, L.rows, S, 16);
    st.same = alike(L.x, L.ldx, L.residual, L.ldr, L.rows, S) && alike(L.x, L.ldx, L.residual_out, L.ldro, L.rows, S);
    st.y_same = st.same && alike(L.x, L.ldx, L.y, L.ldy, L.rows, S);
    const bool vec = L.cols % VEC == 0 && rows_on(L.x, L.ldx, L.rows, S, 16) &&
                     rows_on(L.residual, L.ldr, L.rows, S, 16) && rows_on(L.residual_out, L.ldro, L.rows, S, 16) &&
                     st.w_vec && st.y_vec && st.q_vec;
    int status = GEMM_OK;
    if (vec ? launch_rows<T, VEC>(L, stream, &status) : launch_rows<T, 1>(L, stream, &status)) return status;
    constexpr int64_t kMostStaged = 45000;
    if (L.cols > kMostStaged) return launch(wide_kernel<T>, L.rows, 1024, 0, stream, L);
    const size_t smem = static_cast<size_t>(L.cols + L.cols / 8 + 8) * sizeof(float);
    {
        static std::mutex mu;
        static bool done[64] = {};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GEMM_ERR_CUDA;
        std::lock_guard<std::mutex> g(mu);
        if (!done[dev]) {
            if (cudaFuncSetAttribute(staged_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (kMostStaged + kMostStaged / 8 + 8) * sizeof(float)) != cudaSuccess)
                return GEMM_ERR_LAUNCH;
            done[dev] = true;
        }
    }
    // Few threads a row with more rows an SM until a row fills them: 8000 x 2541
    // bf16 takes 37.4 us with 128 threads and 45.8 with 256, x 5001 72.9 with 128,
    // 65.0 with 192 and 69.9 with 256, x 12001 200 with 256 and 185 with 512.
    const int threads = L.cols >= 7168 || L.rows <= tc_current_device_sms() ? 512
                        : L.cols >= 5376 || sizeof(T) == 4                  ? 256
                        : L.cols >= 2560                                    ? 192 : 128;
    return launch(staged_kernel<T>, L.rows, threads, smem, stream, L, st);
}

}  // namespace

int norm_launch(const NormLaunch& given, cudaStream_t stream) {
    NormLaunch L = given;
    L.inv_cols = L.cols > 0 ? static_cast<float>(1.0 / static_cast<double>(L.cols)) : 0.0f;
    if (L.dtype == QUANT_F32) return launch_type<float>(L, stream);
    if (L.dtype == QUANT_F16) return launch_type<__half>(L, stream);
    return launch_type<__nv_bfloat16>(L, stream);
}

}  // namespace ssp
