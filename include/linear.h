/*
 * linear.h -- C ABI of libgemm.so's operators that train a 16-bit linear layer
 * (sm_103a):
 *
 *   linear         the layer: a product with bias, activation and residual in
 *                  its epilogue
 *   act_grad       the gradient through the activation, and the bias gradient
 *   linear_dx      the gradient of the layer's input, and through the
 *                  activation below it
 *   linear_dw      the gradient of the weights
 *   orthogonalize  a weight's update with all its singular values brought near
 *                  one by Newton-Schulz steps
 *
 * A layer y = act(x W^T + b) + r is differentiated by
 *
 *     act_grad    dz = dy * act'(z),  db = sum of dz's rows
 *     linear_dx   dx = dz W
 *     linear_dw   dW = dz^T x
 *
 * and dr = dy.  In a stack, linear_dx of one layer may do the next one's
 * act_grad as well (its `act` and `pre`).
 *
 * Memory, streams and errors are gemm.h's: all pointers are device pointers
 * owned by the caller, no pointer is kept after a call, nothing is allocated,
 * `stream` is a cudaStream_t (NULL = the legacy default stream), every entry
 * point but those that end in _checked and those that are host code alone
 * (linear_plan, orthogonalize_workspace) enqueues its work and returns without
 * synchronising, and gives a gemm_status_t.  Argument checks are made on the
 * host before anything is enqueued.  Leading dimensions are in elements and may
 * exceed the row length; a single row's leading dimension is not looked at.
 * Outputs must not overlap inputs or each other unless an entry point says so.
 * Rows, columns, M, N and K above 2^31 - 4097 are GEMM_ERR_UNSUPPORTED.  Every
 * result is the same, bit for bit, from call to call.
 *
 * 16-bit tensors are fp16 or bf16 (`dtype`: QUANT_F16 or QUANT_BF16 of quant.h;
 * QUANT_F32 is GEMM_ERR_UNSUPPORTED where 16 bits are asked for).  Products are
 * summed in fp32 on the tensor cores, everything after the sum is fp32, and
 * each output is rounded once (fp16 overflows to infinity).
 *
 * Alignment (GEMM_ERR_ALIGN otherwise): matrices start on 16-byte boundaries
 * and their leading dimensions are multiples of 16 bytes, act_grad's excepted;
 * vectors are aligned to their element.  Rows that start on 128-byte lines are the
 * fast case of the products.
 */
#ifndef SSP_LINEAR_H
#define SSP_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"
#include "quant.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Activations and their derivatives.  At infinities both are their limits
 * (those of -infinity are 0, to within 3e-17), and a NaN gives a NaN, but relu's
 * derivative, which is 1 there.  relu'(0) = 0.
 */
typedef enum {
    LINEAR_ACT_NONE = 0,
    LINEAR_ACT_RELU = 1,      /* max(z, 0) */
    LINEAR_ACT_GELU = 2,      /* z Phi(z), Phi the normal distribution function */
    LINEAR_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    LINEAR_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} linear_act_t;

/* The kernels of the products, as linear_plan names them. */
typedef enum {
    LINEAR_KERNEL_FEW = 0, /* tiles of 128 columns by 16 to 256 rows, K cut over a cluster */
    LINEAR_KERNEL_PAIR = 1 /* tiles of 256 rows by 192 to 256 columns on CTA pairs */
} linear_kernel_t;

/* The products whose launch linear_plan tells. */
typedef enum {
    LINEAR_OP_FORWARD = 0, /* linear:    M x N results, sums of K */
    LINEAR_OP_DX = 1,      /* linear_dx: M x K results, sums of N */
    LINEAR_OP_DW = 2       /* linear_dw: N x K results, sums of M */
} linear_op_t;

/*
 * linear -- z = x W^T + bias, y = act(z) + residual
 *   x         M x K, ldx >= K
 *   W         N x K (a row an output), ldw >= K
 *   bias      N values of the same type, or NULL
 *   residual  M x N, ldr >= N, or NULL; may be the same buffer as y (same
 *             leading dimension)
 *   pre       M x N, ldp >= N: receives z, which act_grad and linear_dx read;
 *             or NULL
 *   y         M x N, ldy >= N
 * All of one 16-bit type.  The activation is applied to the unrounded z.
 * K = 0 gives z = bias.
 */
int linear(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W, int64_t ldw,
           const void* bias, const void* residual, int64_t ldr, int act, void* pre, int64_t ldp,
           void* y, int64_t ldy, int dtype, void* stream);

/*
 * act_grad -- dz = dy * act'(pre), dbias = addend + the sum of dz's rows
 *   dy, pre   M x N of one 16-bit type; pre may be NULL for LINEAR_ACT_NONE
 *   dz        M x N of that type; may be dy or pre itself (same leading
 *             dimension), or NULL (not computed)
 *   dbias     N fp32 values, or NULL (not computed); the sum takes the
 *             unrounded dz in a fixed order.  M = 0 gives the addend.
 *   addend    N fp32 values, or NULL (zeros); may be dbias itself
 * dz and dbias are not both NULL.  No alignment is asked for beyond the
 * element's own; rows on 16-byte boundaries are the fast case.
 */
int act_grad(int64_t M, int64_t N, const void* dy, int64_t lddy, const void* pre, int64_t ldp,
             int act, void* dz, int64_t lddz, float* dbias, const float* addend, int dtype,
             void* stream);

/*
 * linear_dx -- dx = (dz W + residual) * act'(pre)
 *   dz        M x N, lddz >= N
 *   W         N x K, ldw >= K
 *   residual  M x K, ldr >= K: a gradient that arrives by another way, added
 *             before the derivative is applied; or NULL
 *   pre       M x K, ldp >= K: what the activation that made the layer's input
 *             was applied to; NULL (and only then) for LINEAR_ACT_NONE
 *   dx        M x K, lddx >= K; may be the same buffer as residual or pre (same
 *             leading dimension)
 * All of one 16-bit type.  N = 0 gives a sum of 0.
 */
int linear_dx(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* W,
              int64_t ldw, const void* residual, int64_t ldr, int act, const void* pre,
              int64_t ldp, void* dx, int64_t lddx, int dtype, void* stream);

/*
 * linear_dw -- dW = dz^T x + addend
 *   dz        M x N, lddz >= N;  x  M x K, ldx >= K: of one 16-bit type
 *   dW        N x K of out_dtype: QUANT_F32 or `dtype`; lddw >= K
 *   addend    N x K of out_dtype, ldc >= K, or NULL; may be dW itself (same
 *             leading dimension)
 * With an fp32 dW, no accumulator of the tensor cores, which truncate as they add, sums
 * more than 512 rows (in large ones two of a sum 1024): a dW of any number of rows is
 * about as good as by fp32 sums.  (A
 * 16-bit dW is summed by one accumulator, which loses up to 6e-9 of the sum of
 * magnitudes a row: half an fp16 step at 80000 rows of equal signs.)
 * M = 0 gives the addend (or 0).
 */
int linear_dw(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* x,
              int64_t ldx, const void* addend, int64_t ldc, void* dW, int64_t lddw, int dtype,
              int out_dtype, void* stream);

/*
 * linear_checked, linear_dx_checked, linear_dw_checked -- the same, then
 * synchronise `stream` and read (and clear) the product kernels' device status
 * word: GEMM_ERR_TIMEOUT if a pipeline wait ran out (the output is then
 * undefined; gemm_debug_set's hooks apply), GEMM_ERR_CUDA if the stream
 * reported an error.  Meant for tests and debugging.
 */
int linear_checked(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
                   int64_t ldw, const void* bias, const void* residual, int64_t ldr, int act,
                   void* pre, int64_t ldp, void* y, int64_t ldy, int dtype, void* stream);
int linear_dx_checked(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* W,
                      int64_t ldw, const void* residual, int64_t ldr, int act, const void* pre,
                      int64_t ldp, void* dx, int64_t lddx, int dtype, void* stream);
int linear_dw_checked(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* x,
                      int64_t ldx, const void* addend, int64_t ldc, void* dW, int64_t lddw,
                      int dtype, int out_dtype, void* stream);

/*
 * linear_plan -- the launch one of the products (`op`: a linear_op_t) would
 * make for these sizes, without making it; out_dtype is the output's type.  (A
 * residual or addend may take the room of some of the ring's stages.)  The
 * plan's kernel is a linear_kernel_t.  Needs a current CUDA device.
 * GEMM_ERR_ARG for sizes below 1, an unknown op or dtype or a NULL plan;
 * GEMM_ERR_UNSUPPORTED as the products.
 */
int linear_plan(int op, int64_t M, int64_t N, int64_t K, int out_dtype, quant_plan_t* plan);

/*
 * orthogonalize -- for each of `batch` matrices G (rows x cols)
 *
 *     X = G / (|G| + eps)                    (|G|: the root of the sum of squares)
 *     `steps` times:  A = X X^T,  X = a X + (b A + c A^2) X
 *     out = scale * X
 *
 * which brings the singular values of G near one (to 0.65 .. 1.25 in five steps
 * with a, b, c = 3.4445, -4.7750, 2.0315, but for those below 2e-3 |G|) and
 * leaves its singular vectors.  A matrix of more rows than columns takes
 * A = X^T X and X (...) instead, which gives the same.
 *   g          batch matrices, `stride_g` elements apart, of any quant_type_t,
 *              ldg >= cols
 *   out        likewise; out_dtype QUANT_F16 or QUANT_BF16
 *   coefficients  a, b and c (host memory)
 *   steps      0 .. 100
 *   workspace  orthogonalize_workspace(...) bytes (GEMM_ERR_SCRATCH if
 *              workspace_bytes is less) on a 256-byte boundary, whose
 *              contents need not be kept from call to call; calls that may run
 *              at the same time (captured graphs among them) each need their own
 * X, A and b A + c A^2 are held in fp16 between the products, at power-of-two
 * scales that put their elements in fp16's range; the products are summed and
 * combined in fp32.  That is 2^-11 a rounding, an eighth of what bf16 would
 * lose: in five steps a gradient of full rank comes out within 2e-3 of its norm
 * where its shorter side is 100 or more, 4e-3 from 9 on and 1e-2 below (a step makes
 * an error beside a singular value of 1.2 four times as large; many of them average),
 * before the output's own rounding.  Directions whose singular value is below some
 * 1e-4 |G| are lost in the roundings, as is a G that is small beside eps.  The
 * scales hold for coefficients that keep X's singular values below 1.9 and those of
 * b A + c A^2 below 3.9; others may overflow to infinity.  A NaN or an infinity in a
 * matrix makes its output NaN; a matrix of zeros gives zeros (with eps = 0: NaN).
 * Elements of every finite magnitude are taken.  rows and cols above 32768 are
 * GEMM_ERR_UNSUPPORTED, as is a batch above 65535.  The strides between
 * matrices are multiples of 16 bytes (not looked at for a single matrix).
 */
int orthogonalize(int64_t batch, int64_t rows, int64_t cols, const void* g, int64_t ldg,
                  int64_t stride_g, int dtype, void* out, int64_t ldo, int64_t stride_o,
                  int out_dtype, int steps, const float* coefficients, float eps, float scale,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * orthogonalize_checked -- orthogonalize as linear_checked is linear.  (Matrices with a
 * side of 128 at most may take one launch, in which gemm_debug_set's withhold_arrive is
 * the number of the product, three a step, whose end the first CTA is not told of.)
 */
int orthogonalize_checked(int64_t batch, int64_t rows, int64_t cols, const void* g, int64_t ldg,
                          int64_t stride_g, int dtype, void* out, int64_t ldo, int64_t stride_o,
                          int out_dtype, int steps, const float* coefficients, float eps,
                          float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that orthogonalize needs (*bytes); 0 for empty matrices. */
int orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* SSP_LINEAR_H */
