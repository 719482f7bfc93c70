// quant.h -- launcher interfaces shared by the quantised operators' C ABI
// (quant_api.cu) and their kernels.  Not installed; the public interface is
// include/quant.h.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/quant.h"

namespace ssp {

struct GemmDeviceStatus;

// One row-wise pass: the residual's addition, the norm and the 8-bit rows
// (rmsnorm.cu).  Null pointers are inputs that are absent and outputs that
// are not wanted; weight == nullptr: no norm (y = h).
struct NormLaunch {
    int64_t rows, cols;
    const void* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    const void* weight;
    float eps;
    int dtype;  // quant_type_t
    void* residual_out;
    int64_t ldro;
    void* y;
    int64_t ldy;
    void* q;
    int64_t ldq;
    float* scale;
    float inv_cols;  // 1/cols, set by norm_launch
};
int norm_launch(const NormLaunch& L, cudaStream_t stream);

// e4m3 product (gemm_fp8_sm103a.cu); M, N, K > 0.
struct Fp8Launch {
    int64_t M, N, K;
    const void* A;
    int64_t lda;
    const void* B;
    int64_t ldb;
    void* C;
    int64_t ldc;
    const float* a_scale;
    const float* b_scale;
    int out_bf16;  // 0 fp16, 1 bf16
    quant_plan_t* plan = nullptr;  // filled instead of launching, if given
};
int fp8_launch(const Fp8Launch& L, cudaStream_t stream);
// The fp8 kernels' device status word, read and reset (synchronous).
int fp8_read_and_clear_status(GemmDeviceStatus* out);

// 4-bit weights (gemv_w4.cu); M, N, K > 0.
struct W4Launch {
    int64_t M, N, K;
    const void* x;
    int64_t ldx;
    const uint8_t* W;
    int64_t ldw;
    const void* scales;
    int64_t lds;
    const uint8_t* zeros;
    int64_t ldz;
    int group;
    void* C;
    int64_t ldc;
    int bf16;  // 0 fp16, 1 bf16
    quant_plan_t* plan = nullptr;  // filled instead of launching, if given
};
int w4_launch(const W4Launch& L, cudaStream_t stream);
int w4_read_and_clear_status(GemmDeviceStatus* out);

struct W4QuantLaunch {
    int64_t N, K;
    const void* w;
    int64_t ld;
    int dtype;
    int group;
    uint8_t* W;
    int64_t ldw;
    void* scales;
    int64_t lds;
    int scale_bf16;
    uint8_t* zeros;
    int64_t ldz;
};
int w4_quantize_launch(const W4QuantLaunch& L, cudaStream_t stream);

}  // namespace ssp
