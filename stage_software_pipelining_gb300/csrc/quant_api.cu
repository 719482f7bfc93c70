// quant_api.cu -- the C ABI of the quantised operators (declared in
// include/quant.h): argument checks, degenerate sizes and dispatch.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/quant.h"
#include "internal.h"
#include "quant.h"

namespace {

// Largest rows and columns: indices of a last tile's end stay 32-bit integers.
constexpr int64_t kMost = INT_MAX - 4096;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool known(int dtype) { return dtype >= QUANT_F32 && dtype <= QUANT_BF16; }
int size_of(int dtype) { return dtype == QUANT_F32 ? 4 : 2; }

// A leading dimension is looked at where there is a second row to reach.
bool ld_ok(int64_t rows, int64_t ld, int64_t cols) { return rows <= 1 || ld >= cols; }

int norm_checked(ssp::NormLaunch L, void* stream) {
    if (L.rows < 0 || L.cols < 0 || !known(L.dtype)) return GEMM_ERR_ARG;
    if (L.cols > 0) {  // buffers without elements may have no address
        if ((L.q == nullptr) != (L.scale == nullptr)) return GEMM_ERR_ARG;
        if (!L.residual_out && !L.y && !L.q) return GEMM_ERR_ARG;
    }
    if (!(L.eps >= 0.0f)) return GEMM_ERR_ARG;
    if (L.rows == 0) return GEMM_OK;
    if (L.rows > kMost || L.cols > kMost) return GEMM_ERR_UNSUPPORTED;
    if (L.cols == 0 && L.scale == nullptr) return GEMM_OK;
    if (L.cols > 0 && L.x == nullptr) return GEMM_ERR_ARG;
    const uintptr_t es = static_cast<uintptr_t>(size_of(L.dtype));
    if (!ld_ok(L.rows, L.ldx, L.cols)) return GEMM_ERR_ARG;
    if (L.residual && !ld_ok(L.rows, L.ldr, L.cols)) return GEMM_ERR_ARG;
    if (L.residual_out && !ld_ok(L.rows, L.ldro, L.cols)) return GEMM_ERR_ARG;
    if (L.y && !ld_ok(L.rows, L.ldy, L.cols)) return GEMM_ERR_ARG;
    if (L.q && !ld_ok(L.rows, L.ldq, L.cols)) return GEMM_ERR_ARG;
    for (const void* p : {L.x, L.residual, L.weight, static_cast<const void*>(L.residual_out),
                          static_cast<const void*>(L.y)})
        if (!aligned(p, es)) return GEMM_ERR_ALIGN;
    if (!aligned(L.scale, 4)) return GEMM_ERR_ALIGN;
    return ssp::norm_launch(L, static_cast<cudaStream_t>(stream));
}

// After a launch: wait for the stream and look at the kernels' status word.
int checked(int (*status)(ssp::GemmDeviceStatus*), void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
    ssp::GemmDeviceStatus ds;
    const int st = status(&ds);
    if (st != GEMM_OK) return st;
    return ds.code != 0 ? GEMM_ERR_TIMEOUT : GEMM_OK;
}

}  // namespace

extern "C" {

int add_rmsnorm(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual,
                int64_t ldr, const void* weight, float eps, int dtype, void* residual_out,
                int64_t ldro, void* y, int64_t ldy, void* q, int64_t ldq, float* scale,
                void* stream) {
    if (weight == nullptr && rows > 0 && cols > 0) return GEMM_ERR_ARG;
    // Rows without elements have no mean to divide by, only the least scale.
    return norm_checked({rows, cols, x, ldx, residual, ldr, cols > 0 ? weight : nullptr, eps, dtype, residual_out, ldro, y,
                         ldy, q, ldq, scale},
                        stream);
}

int quantize_fp8(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, void* q,
                 int64_t ldq, float* scale, void* stream) {
    if (rows > 0 && ((q == nullptr && cols > 0) || scale == nullptr)) return GEMM_ERR_ARG;
    if (rows == 0 && cols >= 0 && known(dtype)) return GEMM_OK;
    return norm_checked({rows, cols, x, ldx, nullptr, 0, nullptr, 0.0f, dtype, nullptr, 0, nullptr,
                         0, q, ldq, scale},
                        stream);
}

int gemm_fp8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
             int64_t ldb, void* C, int64_t ldc, const float* a_scale, const float* b_scale,
             int dtype, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !known(dtype)) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (C == nullptr || !ld_ok(M, ldc, N)) return GEMM_ERR_ARG;
    if (K > 0 && (A == nullptr || B == nullptr || a_scale == nullptr || b_scale == nullptr))
        return GEMM_ERR_ARG;
    if (K > 0 && (!ld_ok(M, lda, K) || !ld_ok(N, ldb, K))) return GEMM_ERR_ARG;
    if (M > kMost || N > kMost || K > kMost) return GEMM_ERR_UNSUPPORTED;
    // A single row's leading dimension is never used, but the tensor maps
    // hold one: the row length on a 16-byte boundary.
    if (M <= 1) lda = (K + 15) / 16 * 16;
    if (N <= 1) ldb = (K + 15) / 16 * 16;
    if (M <= 1) ldc = (N + 7) / 8 * 8;
    if (!aligned(C, 16) || (ldc * 2) % 16 != 0) return GEMM_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return ssp::scale_launch(M, N, C, ldc, 1, 0.0f, s);  // 16-bit zeros
    if (!aligned(A, 16) || !aligned(B, 16) || lda % 16 != 0 || ldb % 16 != 0) return GEMM_ERR_ALIGN;
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4)) return GEMM_ERR_ALIGN;
    return ssp::fp8_launch({M, N, K, A, lda, B, ldb, C, ldc, a_scale, b_scale, dtype == QUANT_BF16}, s);
}

int gemm_fp8_checked(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                     int64_t ldb, void* C, int64_t ldc, const float* a_scale, const float* b_scale,
                     int dtype, void* stream) {
    const int st = gemm_fp8(M, N, K, A, lda, B, ldb, C, ldc, a_scale, b_scale, dtype, stream);
    return st != GEMM_OK ? st : checked(ssp::fp8_read_and_clear_status, stream);
}

int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int dtype, quant_plan_t* plan) {
    if (M < 1 || N < 1 || K < 1 || !known(dtype) || plan == nullptr) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32 || M > kMost || N > kMost || K > kMost) return GEMM_ERR_UNSUPPORTED;
    ssp::Fp8Launch L{};
    L.M = M;
    L.N = N;
    L.K = K;
    L.out_bf16 = dtype == QUANT_BF16;
    L.plan = plan;
    return ssp::fp8_launch(L, nullptr);
}

int gemv_w4(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
            int64_t ldw, const void* scales, int64_t lds, const void* zeros, int64_t ldz,
            int group, void* C, int64_t ldc, int dtype, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !known(dtype)) return GEMM_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_ERR_ARG;
    if (K % group != 0) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (C == nullptr || !ld_ok(M, ldc, N)) return GEMM_ERR_ARG;
    const int64_t groups = K / group;
    if (K > 0 && (x == nullptr || W == nullptr || scales == nullptr)) return GEMM_ERR_ARG;
    if (K > 0 && (!ld_ok(M, ldx, K) || !ld_ok(N, ldw, K / 2) || !ld_ok(N, lds, groups)))
        return GEMM_ERR_ARG;
    if (K > 0 && zeros && !ld_ok(N, ldz, groups)) return GEMM_ERR_ARG;
    if (M > kMost || N > kMost || K > (1 << 26)) return GEMM_ERR_UNSUPPORTED;
    if (N <= 1) lds = ldz = groups;
    if (lds > (1 << 22) || (zeros && ldz > (1 << 22))) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(C, 2)) return GEMM_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return ssp::scale_launch(M, N, C, ldc, 1, 0.0f, s);  // 16-bit zeros
    if (M <= 1) ldx = K;
    if (N <= 1) ldw = K / 2;
    if (!aligned(x, 16) || (ldx * 2) % 16 != 0) return GEMM_ERR_ALIGN;
    if (!aligned(W, 16) || ldw % 16 != 0) return GEMM_ERR_ALIGN;
    if (!aligned(scales, 2)) return GEMM_ERR_ALIGN;
    return ssp::w4_launch({M, N, K, x, ldx, static_cast<const uint8_t*>(W), ldw, scales, lds,
                           static_cast<const uint8_t*>(zeros), ldz, group, C, ldc,
                           dtype == QUANT_BF16},
                          s);
}

int gemv_w4_checked(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
                    int64_t ldw, const void* scales, int64_t lds, const void* zeros, int64_t ldz,
                    int group, void* C, int64_t ldc, int dtype, void* stream) {
    const int st = gemv_w4(M, N, K, x, ldx, W, ldw, scales, lds, zeros, ldz, group, C, ldc, dtype, stream);
    return st != GEMM_OK ? st : checked(ssp::w4_read_and_clear_status, stream);
}

int gemv_w4_plan(int64_t M, int64_t N, int64_t K, int group, int zeros, int dtype, quant_plan_t* plan) {
    if (M < 1 || N < 1 || K < 1 || !known(dtype) || plan == nullptr) return GEMM_ERR_ARG;
    if ((group != 32 && group != 64 && group != 128) || K % group != 0 || (zeros != 0 && zeros != 1))
        return GEMM_ERR_ARG;
    if (dtype == QUANT_F32 || M > kMost || N > kMost || K > (1 << 26)) return GEMM_ERR_UNSUPPORTED;
    ssp::W4Launch L{};
    L.M = M;
    L.N = N;
    L.K = K;
    L.group = group;
    // The choice asks whether there are zero points, not what they are.
    L.zeros = zeros ? reinterpret_cast<const uint8_t*>(static_cast<uintptr_t>(256)) : nullptr;
    L.bf16 = dtype == QUANT_BF16;
    L.plan = plan;
    return ssp::w4_launch(L, nullptr);
}

int quantize_w4(int64_t N, int64_t K, const void* w, int64_t ld, int dtype, int group, void* W,
                int64_t ldw, void* scales, int64_t lds, int scale_dtype, void* zeros, int64_t ldz,
                void* stream) {
    if (N < 0 || K < 0 || !known(dtype) || !known(scale_dtype)) return GEMM_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_ERR_ARG;
    if (K % group != 0) return GEMM_ERR_ARG;
    if (scale_dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return GEMM_OK;
    const int64_t groups = K / group;
    if (w == nullptr || W == nullptr || scales == nullptr) return GEMM_ERR_ARG;
    if (!ld_ok(N, ld, K) || !ld_ok(N, ldw, K / 2) || !ld_ok(N, lds, groups)) return GEMM_ERR_ARG;
    if (zeros && !ld_ok(N, ldz, groups)) return GEMM_ERR_ARG;
    if (N > kMost || K > (1 << 26)) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(w, static_cast<uintptr_t>(size_of(dtype))) || !aligned(scales, 2)) return GEMM_ERR_ALIGN;
    return ssp::w4_quantize_launch({N, K, w, ld, dtype, group, static_cast<uint8_t*>(W), ldw, scales,
                                    lds, scale_dtype == QUANT_BF16, static_cast<uint8_t*>(zeros), ldz},
                                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
