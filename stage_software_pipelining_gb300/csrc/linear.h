// linear.h -- launcher interfaces shared by the training operators' C ABI
// (linear_api.cu) and their kernels.  Not installed; the public interface is
// include/linear.h.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/linear.h"

namespace ssp {

struct GemmDeviceStatus;

// What a product's epilogue does with a sum (acc) of its output element (i, j).
enum ProductEpilogue {
    EPI_LINEAR = 0,  // z = acc + bias_j (kept in P if given); act(z) + R
    EPI_GRAD = 1,    // (acc + R) * act'(P)
    EPI_F32 = 2,     // acc + R, fp32 R and output
    EPI_STEP = 3     // alpha * acc + beta * R, fp16 operands and R
};

// One matrix of a product: element (r, c) of matrix b at
// p[b * stride + r * ld + c].
struct ProductMatrix {
    const void* p = nullptr;
    int64_t ld = 0;
    int64_t stride = 0;
};

// D = epilogue(A B) for `batch` products of M x N results and sums of K; M, N >
// 0, K >= 0.  A is stored M x K, or K x M where a_mn is set; B is stored N x K, or
// K x N where b_mn is set.
struct ProductLaunch {
    int64_t M, N, K, batch = 1;
    ProductMatrix A, B;
    int a_mn = 0, b_mn = 0;
    int bf16 = 0;  // operands: 0 fp16, 1 bf16
    int epi = EPI_LINEAR;
    int act = 0;
    ProductMatrix D;       // the output
    int out_bf16 = 0;      // a 16-bit output's type
    const void* bias = nullptr;
    ProductMatrix R, P;
    float alpha = 1.0f, beta = 1.0f;  // EPI_STEP
    // EPI_STEP, or null: a factor t per matrix on the device; alpha is
    // multiplied by t^alpha_pow and beta by t^beta_pow.
    const float* factor = nullptr;
    int alpha_pow = 0, beta_pow = 0;
    int symmetric = 0;     // EPI_STEP: D is known to be symmetric (M = N)
    // EPI_STEP: the output's rows are padded to a multiple of 8 elements that
    // may be written.
    int padded = 0;
    quant_plan_t* plan = nullptr;  // filled instead of launching, if given
};
// Chooses a kernel and enqueues it; a gemm_status_t.
int product_launch(const ProductLaunch& L, cudaStream_t stream);
// The product kernels' device status words, read and reset (synchronous).
int product_read_and_clear_status(GemmDeviceStatus* out);

// product_few_sm103a.cu and product_pair_sm103a.cu
int product_few_launch(const ProductLaunch& L, int mt, int split, bool two, cudaStream_t stream);
int product_pair_launch(const ProductLaunch& L, int bn, cudaStream_t stream);
// CTA pairs that the current device holds at once.
int product_resident_pairs();
// CTAs (one an SM) that the current device holds at once, by cluster size 1..8.
bool product_resident_ctas(int (&out)[9]);
int product_few_status(GemmDeviceStatus* out);
int product_pair_status(GemmDeviceStatus* out);

// fp32 outputs: K blocks of 64 that one accumulator sums, 512 rows (a pair tile's first two
// accumulations may have twice as many).  The tensor cores truncate as they add, and
// accumulations join in registers, rounded to nearest: 32768 rows of fp16 come out 6.5e-7
// of the norm off, as by fp32 sums (5.7e-7); with 1024 rows an accumulator 1.3e-6, with
// 4096 4.9e-6.  (32768 x 1024^2 58.0 us for 57.4 with 1024 and 56.3 with 4096.)
constexpr int kProductChunk = 8;

struct ActGradLaunch {
    int64_t M, N;
    const void* dy;
    int64_t lddy;
    const void* pre;
    int64_t ldp;
    int act;
    void* dz;
    int64_t lddz;
    float* dbias;
    const float* addend;
    int bf16;
};
int act_grad_launch(const ActGradLaunch& L, cudaStream_t stream);

struct OrthoLaunch {
    int64_t batch, rows, cols;
    const void* g;
    int64_t ldg, stride_g;
    int dtype;  // quant_type_t
    void* out;
    int64_t ldo, stride_o;
    int out_bf16;
    int steps;
    float a, b, c, eps, scale;
    void* workspace;
};
size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols);
int ortho_launch(const OrthoLaunch& L, cudaStream_t stream);
// Matrices with a short side, all steps in one launch (orthogonalize_small.cu).
bool ortho_small_takes(const OrthoLaunch& L);
int ortho_small_launch(const OrthoLaunch& L, cudaStream_t stream);
int ortho_small_status(GemmDeviceStatus* out);

}  // namespace ssp
