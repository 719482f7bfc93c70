// rmsnorm.cu -- the residual's addition, the root-mean-square norm and the
// 8-bit rows with a scale each, in one kernel:
//
//     h = x + residual,  y = h / sqrt(mean(h^2) + eps) * w,
//     scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
//
// The sums are fp32, and y is never rounded before it is quantised.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/quant.h"
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

template <typename Op>
__device__ __forceinline__ float block_reduce(float v, Op op, float* buf) {
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) v = op(v, buf[w]);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(256) norm_kernel(const NormLaunch p) {
    __shared__ float buf[32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const T* w = static_cast<const T*>(p.weight);
    auto h_at = [&](int i) {
        float h = to_f32(x[i]);
        if (r) h += to_f32(r[i]);
        return h;
    };
    const int n = static_cast<int>(p.cols);
    float rstd = 1.0f;
    if (w) {
        float ss = 0.0f;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const float h = h_at(i);
            ss = fmaf(h, h, ss);
        }
        ss = block_reduce(ss, [](float a, float b) { return a + b; }, buf);
        rstd = rsqrtf(ss / static_cast<float>(n) + p.eps);
    }
    float scale = kScaleMin;
    if (p.scale) {
        float am = 0.0f;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const float y = w ? h_at(i) * rstd * to_f32(w[i]) : h_at(i);
            am = max_nan(am, fabsf(y));
        }
        am = block_reduce(am, [](float a, float b) { return max_nan(a, b); }, buf);
        scale = max_nan(am / kE4m3Max, kScaleMin);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
    const float inv = 1.0f / scale;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const float h = h_at(i);
        const float y = w ? h * rstd * to_f32(w[i]) : h;
        if (p.residual_out) static_cast<T*>(p.residual_out)[row * p.ldro + i] = from_f32<T>(h);
        if (p.y) static_cast<T*>(p.y)[row * p.ldy + i] = from_f32<T>(y);
        if (p.scale)
            static_cast<uint8_t*>(p.q)[row * p.ldq + i] =
                __nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
    }
}

}  // namespace

int norm_launch(const NormLaunch& L, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(L.rows);
    if (L.dtype == QUANT_F32) norm_kernel<float><<<grid, 256, 0, stream>>>(L);
    else if (L.dtype == QUANT_F16) norm_kernel<__half><<<grid, 256, 0, stream>>>(L);
    else norm_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(L);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace ssp
