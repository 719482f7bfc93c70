// linear_api.cu -- the C ABI of the training operators (declared in
// include/linear.h): argument checks, degenerate sizes and dispatch.
#include <cuda_runtime.h>

#include <climits>
#include <initializer_list>
#include <cstdint>

#include "../../include/linear.h"
#include "internal.h"
#include "linear.h"

namespace {

// Largest rows and columns: indices of a last tile's end stay 32-bit integers.
constexpr int64_t kMost = INT_MAX - 4096;
constexpr int64_t kOrthoMost = 32768;  // where the scales of orthogonalize's fp16 tensors were laid out

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool known(int dtype) { return dtype >= QUANT_F32 && dtype <= QUANT_BF16; }
bool known_act(int act) { return act >= LINEAR_ACT_NONE && act <= LINEAR_ACT_SILU; }
int size_of(int dtype) { return dtype == QUANT_F32 ? 4 : 2; }

// A leading dimension is looked at where there is a second row to reach.
bool ld_ok(int64_t rows, int64_t ld, int64_t cols) { return rows <= 1 || ld >= cols; }

// A tensor copy's matrix: on a 16-byte boundary, and its rows.
bool copied_ok(const void* p, int64_t rows, int64_t ld, int size) {
    return aligned(p, 16) && (rows <= 1 || ld * size % 16 == 0);
}

// After a launch: wait for the stream and look at the kernels' status words.
int checked(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
    ssp::GemmDeviceStatus ds;
    const int st = ssp::product_read_and_clear_status(&ds);
    if (st != GEMM_OK) return st;
    return ds.code != 0 ? GEMM_ERR_TIMEOUT : GEMM_OK;
}

// A product's matrices are there, long enough and within the sizes.  Empty
// results are the caller's to return.
struct Given {
    const void* p;
    int64_t rows, cols, ld;
    int size;
    bool needed;
};
int matrices_ok(std::initializer_list<Given> all, int64_t M, int64_t N, int64_t K) {
    for (const Given& g : all) {
        if (g.p == nullptr && g.needed) return GEMM_ERR_ARG;
        if (g.p && !ld_ok(g.rows, g.ld, g.cols)) return GEMM_ERR_ARG;
    }
    if (M > kMost || N > kMost || K > kMost) return GEMM_ERR_UNSUPPORTED;
    for (const Given& g : all)
        if (g.p && !copied_ok(g.p, g.rows, g.ld, g.size)) return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

}  // namespace

namespace ssp {

int product_read_and_clear_status(GemmDeviceStatus* out) {
    *out = {0, 0, 0, 0};
    for (auto read : {product_few_status, product_pair_status, ortho_small_status}) {
        GemmDeviceStatus one;
        const int st = read(&one);
        if (st != GEMM_OK) return st;
        if (one.code != 0) *out = one;
    }
    return GEMM_OK;
}

}  // namespace ssp

extern "C" {

int linear(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W, int64_t ldw,
           const void* bias, const void* residual, int64_t ldr, int act, void* pre, int64_t ldp,
           void* y, int64_t ldy, int dtype, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !known(dtype) || !known_act(act)) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    const int st = matrices_ok({{y, M, N, ldy, 2, true},
                                {K > 0 ? x : nullptr, M, K, ldx, 2, K > 0},
                                {K > 0 ? W : nullptr, N, K, ldw, 2, K > 0},
                                {residual, M, N, ldr, 2, false},
                                {pre, M, N, ldp, 2, false}},
                               M, N, K);
    if (st != GEMM_OK) return st;
    if (!aligned(bias, 2)) return GEMM_ERR_ALIGN;
    ssp::ProductLaunch L;
    L.M = M;
    L.N = N;
    L.K = K;
    L.A = {x, ldx, 0};
    L.B = {W, ldw, 0};
    L.bf16 = L.out_bf16 = dtype == QUANT_BF16;
    L.epi = ssp::EPI_LINEAR;
    L.act = act;
    L.bias = bias;
    L.R = {residual, ldr, 0};
    L.P = {pre, ldp, 0};
    L.D = {y, ldy, 0};
    return ssp::product_launch(L, static_cast<cudaStream_t>(stream));
}

int linear_checked(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
                   int64_t ldw, const void* bias, const void* residual, int64_t ldr, int act,
                   void* pre, int64_t ldp, void* y, int64_t ldy, int dtype, void* stream) {
    const int st = linear(M, N, K, x, ldx, W, ldw, bias, residual, ldr, act, pre, ldp, y, ldy, dtype, stream);
    return st != GEMM_OK ? st : checked(stream);
}

int act_grad(int64_t M, int64_t N, const void* dy, int64_t lddy, const void* pre, int64_t ldp,
             int act, void* dz, int64_t lddz, float* dbias, const float* addend, int dtype,
             void* stream) {
    if (M < 0 || N < 0 || !known(dtype) || !known_act(act)) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || (M == 0 && dbias == nullptr)) return GEMM_OK;
    if (dz == nullptr && dbias == nullptr) return GEMM_ERR_ARG;
    if (act == LINEAR_ACT_NONE) pre = nullptr;
    if (M > 0) {
        if (dy == nullptr || (pre == nullptr && act != LINEAR_ACT_NONE)) return GEMM_ERR_ARG;
        if (!ld_ok(M, lddy, N) || (pre && !ld_ok(M, ldp, N)) || (dz && !ld_ok(M, lddz, N))) return GEMM_ERR_ARG;
    }
    if (M > kMost || N > kMost) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(dy, 2) || !aligned(pre, 2) || !aligned(dz, 2) || !aligned(dbias, 4) || !aligned(addend, 4))
        return GEMM_ERR_ALIGN;
    return ssp::act_grad_launch({M, N, dy, lddy, pre, ldp, act, dz, lddz, dbias, addend, dtype == QUANT_BF16},
                                static_cast<cudaStream_t>(stream));
}

int linear_dx(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* W,
              int64_t ldw, const void* residual, int64_t ldr, int act, const void* pre,
              int64_t ldp, void* dx, int64_t lddx, int dtype, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !known(dtype) || !known_act(act)) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return GEMM_OK;
    if ((pre == nullptr) != (act == LINEAR_ACT_NONE)) return GEMM_ERR_ARG;
    const int st = matrices_ok({{dx, M, K, lddx, 2, true},
                                {N > 0 ? dz : nullptr, M, N, lddz, 2, N > 0},
                                {N > 0 ? W : nullptr, N, K, ldw, 2, N > 0},
                                {residual, M, K, ldr, 2, false},
                                {pre, M, K, ldp, 2, false}},
                               M, N, K);
    if (st != GEMM_OK) return st;
    ssp::ProductLaunch L;
    L.M = M;
    L.N = K;
    L.K = N;
    L.A = {dz, lddz, 0};
    L.B = {W, ldw, 0};
    L.b_mn = 1;
    L.bf16 = L.out_bf16 = dtype == QUANT_BF16;
    L.epi = act == LINEAR_ACT_NONE ? ssp::EPI_LINEAR : ssp::EPI_GRAD;
    L.act = act;
    L.R = {residual, ldr, 0};
    L.P = {pre, ldp, 0};
    L.D = {dx, lddx, 0};
    return ssp::product_launch(L, static_cast<cudaStream_t>(stream));
}

int linear_dx_checked(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* W,
                      int64_t ldw, const void* residual, int64_t ldr, int act, const void* pre,
                      int64_t ldp, void* dx, int64_t lddx, int dtype, void* stream) {
    const int st = linear_dx(M, N, K, dz, lddz, W, ldw, residual, ldr, act, pre, ldp, dx, lddx, dtype, stream);
    return st != GEMM_OK ? st : checked(stream);
}

int linear_dw(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* x,
              int64_t ldx, const void* addend, int64_t ldc, void* dW, int64_t lddw, int dtype,
              int out_dtype, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !known(dtype) || !known(out_dtype)) return GEMM_ERR_ARG;
    if (dtype == QUANT_F32 || (out_dtype != QUANT_F32 && out_dtype != dtype)) return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return GEMM_OK;
    const int so = size_of(out_dtype);
    const int st = matrices_ok({{dW, N, K, lddw, so, true},
                                {M > 0 ? dz : nullptr, M, N, lddz, 2, M > 0},
                                {M > 0 ? x : nullptr, M, K, ldx, 2, M > 0},
                                {addend, N, K, ldc, so, false}},
                               M, N, K);
    if (st != GEMM_OK) return st;
    ssp::ProductLaunch L;
    L.M = N;
    L.N = K;
    L.K = M;
    L.A = {dz, lddz, 0};
    L.B = {x, ldx, 0};
    L.a_mn = L.b_mn = 1;
    L.bf16 = dtype == QUANT_BF16;
    L.out_bf16 = out_dtype == QUANT_BF16;
    L.epi = out_dtype == QUANT_F32 ? ssp::EPI_F32 : ssp::EPI_LINEAR;
    L.R = {addend, ldc, 0};
    L.D = {dW, lddw, 0};
    return ssp::product_launch(L, static_cast<cudaStream_t>(stream));
}

int linear_dw_checked(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* x,
                      int64_t ldx, const void* addend, int64_t ldc, void* dW, int64_t lddw,
                      int dtype, int out_dtype, void* stream) {
    const int st = linear_dw(M, N, K, dz, lddz, x, ldx, addend, ldc, dW, lddw, dtype, out_dtype, stream);
    return st != GEMM_OK ? st : checked(stream);
}

int linear_plan(int op, int64_t M, int64_t N, int64_t K, int out_dtype, quant_plan_t* plan) {
    if (op < LINEAR_OP_FORWARD || op > LINEAR_OP_DW || M < 1 || N < 1 || K < 1 || !known(out_dtype) || plan == nullptr)
        return GEMM_ERR_ARG;
    if ((op != LINEAR_OP_DW && out_dtype == QUANT_F32) || M > kMost || N > kMost || K > kMost)
        return GEMM_ERR_UNSUPPORTED;
    ssp::ProductLaunch L;
    L.M = op == LINEAR_OP_DW ? N : M;
    L.N = op == LINEAR_OP_FORWARD ? N : K;
    L.K = op == LINEAR_OP_FORWARD ? K : op == LINEAR_OP_DX ? N : M;
    L.a_mn = op == LINEAR_OP_DW;
    L.b_mn = op != LINEAR_OP_FORWARD;
    L.epi = out_dtype == QUANT_F32 ? ssp::EPI_F32 : ssp::EPI_LINEAR;
    L.plan = plan;
    return ssp::product_launch(L, nullptr);
}

int orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
    if (batch < 0 || rows < 0 || cols < 0 || bytes == nullptr) return GEMM_ERR_ARG;
    if (batch > 65535 || rows > kOrthoMost || cols > kOrthoMost) return GEMM_ERR_UNSUPPORTED;
    *bytes = batch && rows && cols ? ssp::ortho_workspace(batch, rows, cols) : 0;
    return GEMM_OK;
}

int orthogonalize(int64_t batch, int64_t rows, int64_t cols, const void* g, int64_t ldg,
                  int64_t stride_g, int dtype, void* out, int64_t ldo, int64_t stride_o,
                  int out_dtype, int steps, const float* coefficients, float eps, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (batch < 0 || rows < 0 || cols < 0 || !known(dtype) || !known(out_dtype)) return GEMM_ERR_ARG;
    if (steps < 0 || steps > 100 || (steps > 0 && coefficients == nullptr) || !(eps >= 0.0f)) return GEMM_ERR_ARG;
    if (out_dtype == QUANT_F32) return GEMM_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_OK;
    if (g == nullptr || out == nullptr || workspace == nullptr) return GEMM_ERR_ARG;
    if (!ld_ok(rows, ldg, cols) || !ld_ok(rows, ldo, cols)) return GEMM_ERR_ARG;
    const int64_t ig = rows > 1 ? ldg : cols, io = rows > 1 ? ldo : cols;
    // Matrices of a batch do not overlap.
    if (batch > 1 && (stride_g < (rows - 1) * ig + cols || stride_o < (rows - 1) * io + cols)) return GEMM_ERR_ARG;
    size_t need = 0;
    const int st = orthogonalize_workspace(batch, rows, cols, &need);
    if (st != GEMM_OK) return st;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH;
    const int sg = size_of(dtype);
    if (!copied_ok(g, rows, ldg, sg) || !copied_ok(out, rows, ldo, 2) || !aligned(workspace, 256)) return GEMM_ERR_ALIGN;
    if (batch > 1 && (stride_g * sg % 16 != 0 || stride_o * 2 % 16 != 0)) return GEMM_ERR_ALIGN;
    ssp::OrthoLaunch L = {};
    L.batch = batch;
    L.rows = rows;
    L.cols = cols;
    L.g = g;
    L.ldg = ig;
    L.stride_g = stride_g;
    L.dtype = dtype;
    L.out = out;
    L.ldo = io;
    L.stride_o = stride_o;
    L.out_bf16 = out_dtype == QUANT_BF16;
    L.steps = steps;
    if (steps > 0) {
        L.a = coefficients[0];
        L.b = coefficients[1];
        L.c = coefficients[2];
    }
    L.eps = eps;
    L.scale = scale;
    L.workspace = workspace;
    return ssp::ortho_launch(L, static_cast<cudaStream_t>(stream));
}

int orthogonalize_checked(int64_t batch, int64_t rows, int64_t cols, const void* g, int64_t ldg,
                          int64_t stride_g, int dtype, void* out, int64_t ldo, int64_t stride_o,
                          int out_dtype, int steps, const float* coefficients, float eps,
                          float scale, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = orthogonalize(batch, rows, cols, g, ldg, stride_g, dtype, out, ldo, stride_o, out_dtype, steps,
                                 coefficients, eps, scale, workspace, workspace_bytes, stream);
    return st != GEMM_OK ? st : checked(stream);
}

}  // extern "C"
