// gemv_w4.cu -- C[i,j] = sum_groups scales[j,g] * sum_{k in g} x[i,k] * (w[j,k] - zeros[j,g])
// with 4-bit weights w, and the kernel that makes them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/quant.h"
#include "quant.h"

namespace ssp {
namespace {

template <typename T>
__device__ __forceinline__ float f32_of(T v);
template <>
__device__ __forceinline__ float f32_of(float v) { return v; }
template <>
__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T of_f32(float v);
template <>
__device__ __forceinline__ __half of_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 of_f32(float v) { return __float2bfloat16_rn(v); }

// One warp an output; a lane takes a byte (two weights) at a time.
template <typename T>
__global__ void __launch_bounds__(256) w4_kernel(const W4Launch p) {
    const long long j = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (j >= p.N) return;
    const uint8_t* W = p.W + j * p.ldw;
    const T* s = static_cast<const T*>(p.scales) + j * p.lds;
    for (long long i = blockIdx.y; i < p.M; i += gridDim.y) {
        const T* x = static_cast<const T*>(p.x) + i * p.ldx;
        float acc = 0.0f;
        for (long long b = lane; b < p.K / 2; b += 32) {
            const long long g = 2 * b / p.group;
            const float z = p.zeros ? static_cast<float>(p.zeros[j * p.ldz + g]) : 8.0f;
            const int v = W[b];
            const float lo = static_cast<float>(v & 15) - z, hi = static_cast<float>(v >> 4) - z;
            acc = fmaf(f32_of(s[g]), fmaf(f32_of(x[2 * b]), lo, f32_of(x[2 * b + 1]) * hi), acc);
        }
        for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) static_cast<T*>(p.C)[i * p.ldc + j] = of_f32<T>(acc);
    }
}

// Eight weights (one 32-bit word) a thread, group/8 threads a group.
template <typename T, typename S>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4QuantLaunch p) {
    const long long words = p.K / 8;
    const long long t = blockIdx.x * 256ll + threadIdx.x;
    const bool in = t < p.N * words;
    // Threads past the end repeat the last word, so that whole warps shuffle.
    const long long u = in ? t : p.N * words - 1;
    const long long j = u / words, k = u % words * 8;
    const T* w = static_cast<const T*>(p.w) + j * p.ld + k;
    float v[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = f32_of(w[e]);
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
    for (int o = p.group / 16; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    S s16 = of_f32<S>(p.zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    if (f32_of(s16) < 1.17549435e-38f) s16 = of_f32<S>(0.0f);  // below 2^-126, 1/scale overflows
    const float s = f32_of(s16);
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    const float z = p.zeros ? fminf(rintf(-lo * inv), 15.0f) : 8.0f;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaxf(rintf(v[e] * inv) + z, 0.0f), 15.0f);
        word |= static_cast<uint32_t>(q) << (4 * e);
    }
    if (!in) return;
    uint8_t* out = p.W + j * p.ldw + k / 2;
    for (int e = 0; e < 4; ++e) out[e] = static_cast<uint8_t>(word >> (8 * e));
    if (k % p.group == 0) {
        static_cast<S*>(p.scales)[j * p.lds + k / p.group] = s16;
        if (p.zeros) p.zeros[j * p.ldz + k / p.group] = static_cast<uint8_t>(z);
    }
}

template <typename T>
void quantize_of(const W4QuantLaunch& L, unsigned grid, cudaStream_t stream) {
    if (L.scale_bf16) w4_quantize_kernel<T, __nv_bfloat16><<<grid, 256, 0, stream>>>(L);
    else w4_quantize_kernel<T, __half><<<grid, 256, 0, stream>>>(L);
}

}  // namespace

int w4_launch(const W4Launch& L, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((L.N + 7) / 8),
                    static_cast<unsigned>(L.M < 65535 ? L.M : 65535));
    if (L.bf16) w4_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(L);
    else w4_kernel<__half><<<grid, 256, 0, stream>>>(L);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int w4_quantize_launch(const W4QuantLaunch& L, cudaStream_t stream) {
    const int64_t blocks = (L.N * (L.K / 8) + 255) / 256;
    if (blocks > 0x7fffffffll) return GEMM_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (L.dtype == QUANT_F32) quantize_of<float>(L, grid, stream);
    else if (L.dtype == QUANT_F16) quantize_of<__half>(L, grid, stream);
    else quantize_of<__nv_bfloat16>(L, grid, stream);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace ssp
