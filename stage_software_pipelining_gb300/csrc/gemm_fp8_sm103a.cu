// gemm_fp8_sm103a.cu -- C[i,j] = a_scale[i] * b_scale[j] * sum_k A[i,k] B[k,j]
// with e4m3 A (row-major) and B (column-major) and a 16-bit C.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/quant.h"
#include "quant.h"

namespace ssp {
namespace {

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// 64 x 64 tile of C, 4 x 4 outputs a thread, 16 of K at a time.
__global__ void __launch_bounds__(256) fp8_tile_kernel(const Fp8Launch p) {
    __shared__ float as[16][65], bs[16][65];
    const uint8_t* A = static_cast<const uint8_t*>(p.A);
    const uint8_t* B = static_cast<const uint8_t*>(p.B);
    const long long i0 = 64ll * blockIdx.y, j0 = 64ll * blockIdx.x;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (long long k0 = 0; k0 < p.K; k0 += 16) {
        for (int e = threadIdx.x; e < 64 * 16; e += 256) {
            const int r = e >> 4, k = e & 15;
            const bool in_k = k0 + k < p.K;
            as[k][r] = in_k && i0 + r < p.M ? e4m3_to_f32(A[(i0 + r) * p.lda + k0 + k]) : 0.0f;
            bs[k][r] = in_k && j0 + r < p.N ? e4m3_to_f32(B[(j0 + r) * p.ldb + k0 + k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b)
                    acc[a][b] = fmaf(as[k][ty + 16 * a], bs[k][tx + 16 * b], acc[a][b]);
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const long long i = i0 + ty + 16 * a, j = j0 + tx + 16 * b;
            if (i >= p.M || j >= p.N) continue;
            const float v = acc[a][b] * p.a_scale[i] * p.b_scale[j];
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.C)[i * p.ldc + j] = __float2bfloat16_rn(v);
            else static_cast<__half*>(p.C)[i * p.ldc + j] = __float2half_rn(v);
        }
}

}  // namespace

int fp8_launch(const Fp8Launch& L, cudaStream_t stream) {
    const int64_t gy = (L.M + 63) / 64, gx = (L.N + 63) / 64;
    if (gy > 65535) return GEMM_ERR_UNSUPPORTED;
    fp8_tile_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), 256, 0, stream>>>(L);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace ssp
