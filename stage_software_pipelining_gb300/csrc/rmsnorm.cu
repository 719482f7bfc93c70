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
// each, longer ones a block; a row that does not fit a block's registers is
// read twice (wide_kernel).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

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

// VEC adjacent elements, moved as one access where VEC > 1.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <int VEC>
__device__ __forceinline__ void store_q(uint8_t* q, const float (&y)[VEC]) {
    if constexpr (VEC == 1) {
        *q = __nv_cvt_float_to_fp8(y[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        alignas(VEC) uint16_t v[VEC / 2];
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
            v[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * e], y[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(v);
        else *reinterpret_cast<uint32_t*>(q) = *reinterpret_cast<const uint32_t*>(v);
    }
}

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
    s = lane < warps ? buf[lane] : Stats{0.0f, 0.0f};
    return warp_join(s);
}

// rstd and scale of a row from its Stats.
__device__ __forceinline__ void row_factors(const NormLaunch& p, Stats s, float& rstd, float& scale) {
    rstd = p.weight ? rsqrtf(s.ss / fmaxf(static_cast<float>(p.cols), 1.0f) + p.eps) : 1.0f;
    scale = max_nan(rstd * s.am / kE4m3Max, kScaleMin);
}

// A row in registers: thread t of the row's `threads` holds packs t, t +
// threads, ..., NCH of them.  WARP: a warp a row, blockDim/32 rows a block;
// otherwise a block a row.
constexpr int max_threads(int elements) { return elements <= 16 ? 1024 : 512; }

template <typename T, int VEC, int NCH, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : max_threads(VEC * NCH)) row_kernel(const NormLaunch p) {
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
    const P* x = reinterpret_cast<const P*>(static_cast<const T*>(p.x) + row * p.ldx);
    const P* r = reinterpret_cast<const P*>(static_cast<const T*>(p.residual) + row * p.ldr);
    const P* w = static_cast<const P*>(p.weight);
    P xv[NCH], rv[NCH], wv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int i = t + c * threads;
        if (i < packs) xv[c] = x[i];
    }
    if (p.residual) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int i = t + c * threads;
            if (i < packs) rv[c] = r[i];
        }
    }
    if (p.weight) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int i = t + c * threads;
            if (i < packs) wv[c] = w[i];
        }
    }
    float h[NCH][VEC];
    Stats s = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        if (t + c * threads < packs) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float v = to_f32(xv[c].v[e]);
                if (p.residual) v += to_f32(rv[c].v[e]);
                h[c][e] = v;
                s.ss = fmaf(v, v, s.ss);
                s.am = max_nan(s.am, fabsf(p.weight ? v * to_f32(wv[c].v[e]) : v));
            }
        }
    }
    s = WARP ? warp_join(s) : block_join(s, buf);
    float rstd, scale;
    row_factors(p, s, rstd, scale);
    if (p.scale && t == 0) p.scale[row] = scale;
    const float inv = 1.0f / scale;
    P* ro = reinterpret_cast<P*>(static_cast<T*>(p.residual_out) + row * p.ldro);
    P* yo = reinterpret_cast<P*>(static_cast<T*>(p.y) + row * p.ldy);
    uint8_t* q = static_cast<uint8_t*>(p.q) + row * p.ldq;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int i = t + c * threads;
        if (i < packs) {
            P o;
            if (p.residual_out) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(h[c][e]);
                ro[i] = o;
            }
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = p.weight ? h[c][e] * rstd * to_f32(wv[c].v[e]) : h[c][e];
            if (p.y) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(y[e]);
                yo[i] = o;
            }
            if (p.q) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] *= inv;
                store_q<VEC>(q + static_cast<long long>(i) * VEC, y);
            }
        }
    }
}

// A row too long for a block's registers: one pass for its Stats, one that
// reads it again and writes.  Every element is read and written by the same
// thread, so outputs may lie over inputs.
template <typename T>
__global__ void __launch_bounds__(1024) wide_kernel(const NormLaunch p) {
    __shared__ Stats buf[32];
    griddep_launch_dependents();
    griddep_wait();
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const T* w = static_cast<const T*>(p.weight);
    const int n = static_cast<int>(p.cols);
    Stats s = {0.0f, 0.0f};
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const float h = to_f32(x[i]) + (r ? to_f32(r[i]) : 0.0f);
        s.ss = fmaf(h, h, s.ss);
        s.am = max_nan(s.am, fabsf(w ? h * to_f32(w[i]) : h));
    }
    s = block_join(s, buf);
    float rstd, scale;
    row_factors(p, s, rstd, scale);
    if (p.scale && threadIdx.x == 0) p.scale[row] = scale;
    const float inv = 1.0f / scale;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const float h = to_f32(x[i]) + (r ? to_f32(r[i]) : 0.0f);
        const float y = w ? h * rstd * to_f32(w[i]) : h;
        if (p.residual_out) static_cast<T*>(p.residual_out)[row * p.ldro + i] = from_f32<T>(h);
        if (p.y) static_cast<T*>(p.y)[row * p.ldy + i] = from_f32<T>(y);
        const float qv[1] = {y * inv};
        if (p.q) store_q<1>(static_cast<uint8_t*>(p.q) + row * p.ldq + i, qv);
    }
}

using Kernel = void (*)(const NormLaunch);

int launch(Kernel k, int64_t grid, int threads, const NormLaunch& L, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, L) == cudaSuccess && cudaGetLastError() == cudaSuccess ? GEMM_OK
                                                                                              : GEMM_ERR_LAUNCH;
}

template <typename T, int VEC>
int launch_rows(const NormLaunch& L, cudaStream_t stream) {
    const int64_t packs = (L.cols + VEC - 1) / VEC;
    if (packs <= 128) {  // a warp a row
        Kernel k = packs <= 32 ? row_kernel<T, VEC, 1, true>
                   : packs <= 64 ? row_kernel<T, VEC, 2, true> : row_kernel<T, VEC, 4, true>;
        return launch(k, (L.rows + 3) / 4, 128, L, stream);
    }
    // A block a row: as many threads as packs where there are few rows (the
    // time is one row's), several packs a thread where rows queue for the SMs.
    constexpr int kMost = VEC == 1 ? 8 : 4;  // 16384 elements a block, 8192 one by one
    const bool few = L.rows <= 2 * tc_current_device_sms();
    int nch = few ? 1 : VEC == 1 ? 8 : 4;
    while (nch <= kMost && packs > static_cast<int64_t>(max_threads(VEC * nch)) * nch) nch *= 2;
    if (nch > kMost) return launch(wide_kernel<T>, L.rows, 1024, L, stream);
    Kernel k = nch == 1   ? row_kernel<T, VEC, 1, false>
               : nch == 2 ? row_kernel<T, VEC, 2, false> : row_kernel<T, VEC, 4, false>;
    if constexpr (VEC == 1)
        if (nch == 8) k = row_kernel<T, 1, 8, false>;
    const int threads = static_cast<int>(((packs + nch - 1) / nch + 31) / 32 * 32);
    return launch(k, L.rows, threads, L, stream);
}

// Whether a matrix's rows all start on `to`-byte boundaries.
bool rows_on(const void* p, int64_t ld, int64_t rows, int64_t size, uintptr_t to) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0 &&
                  (rows <= 1 || (ld * size) % static_cast<int64_t>(to) == 0));
}

template <typename T>
int launch_type(const NormLaunch& L, cudaStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int64_t S = sizeof(T);
    const bool vec = L.cols % VEC == 0 && rows_on(L.x, L.ldx, L.rows, S, 16) &&
                     rows_on(L.residual, L.ldr, L.rows, S, 16) && rows_on(L.weight, 0, 1, S, 16) &&
                     rows_on(L.residual_out, L.ldro, L.rows, S, 16) && rows_on(L.y, L.ldy, L.rows, S, 16) &&
                     rows_on(L.q, L.ldq, L.rows, 1, VEC);
    return vec ? launch_rows<T, VEC>(L, stream) : launch_rows<T, 1>(L, stream);
}

}  // namespace

int norm_launch(const NormLaunch& L, cudaStream_t stream) {
    if (L.dtype == QUANT_F32) return launch_type<float>(L, stream);
    if (L.dtype == QUANT_F16) return launch_type<__half>(L, stream);
    return launch_type<__nv_bfloat16>(L, stream);
}

}  // namespace ssp
