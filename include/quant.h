/*
 * quant.h -- C ABI of libgemm.so's operators for a linear layer whose weights
 * or activations are held in few bits (sm_103a):
 *
 *   add_rmsnorm    the residual's addition and the root-mean-square norm, with
 *                  a 16/32-bit result, an 8-bit one with a scale a row, or both
 *   gemm_fp8       the matrix product of 8-bit activations and 8-bit weights
 *   gemv_w4        a few rows of 16-bit activations times 4-bit weights with a
 *                  scale (and a zero point) a group
 *   quantize_fp8   rows to 8 bits, as add_rmsnorm does, without the norm
 *   quantize_w4    a weight matrix to 4 bits
 *
 * 8-bit values are e4m3 (4 exponent bits, 3 mantissa bits, largest 448, no
 * infinity; 0x7f and 0xff are NaN).
 *
 * Memory, streams and errors are gemm.h's: all pointers are device pointers
 * owned by the caller, no pointer is kept after a call, nothing is allocated,
 * `stream` is a cudaStream_t (NULL = the legacy default stream), every entry
 * point but the two that end in _checked and the two that end in _plan
 * (host code alone) enqueues its work and returns without
 * synchronising, and every entry point gives a gemm_status_t.  Argument checks
 * are made on the host before anything is enqueued.  Leading dimensions are in elements (bytes for the
 * packed 4-bit weights) and may exceed the row length; a single row's leading
 * dimension is not looked at.  Outputs must not overlap inputs or each other
 * unless an entry point says so.  Rows, columns, M, N and K above 2^31 - 4097
 * are GEMM_ERR_UNSUPPORTED.  Every result is the same, bit for bit, from
 * call to call.
 */
#ifndef SSP_QUANT_H
#define SSP_QUANT_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QUANT_F32 = 0,
    QUANT_F16 = 1,
    QUANT_BF16 = 2
} quant_type_t;

/* The kernels of the products, as the plan queries name them. */
typedef enum {
    QUANT_KERNEL_FP8_FEW = 0,  /* gemm_fp8: tiles of 16 to 256 rows of A */
    QUANT_KERNEL_FP8_PAIR = 1, /* gemm_fp8: tiles of 256 rows on CTA pairs */
    QUANT_KERNEL_W4_WARP = 2,  /* gemv_w4: tiles of 8 or 16 rows of x, warp-level products */
    QUANT_KERNEL_W4_TC = 3     /* gemv_w4: tiles of 32 rows of x, tcgen05 */
} quant_kernel_t;

/* A launch that a product would make. */
typedef struct {
    int kernel;     /* a quant_kernel_t */
    int tile_rows;  /* rows of A (of x) a tile */
    int split;      /* CTAs that share a tile's K, a cluster */
    int stages;     /* depth of the operand ring */
    int grid;       /* CTAs */
    int smem_bytes; /* dynamic shared memory a CTA */
} quant_plan_t;

/*
 * add_rmsnorm -- for each of `rows` rows of `cols` elements
 *
 *     h = x + residual                        (h = x without a residual)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *     scale = max(max|y| / 448, 2^-126)
 *     q = e4m3(y / scale)                     (nearest even)
 *
 * in fp32, each output rounded once from the fp32 value: residual_out is h,
 * and the norm goes on from the unrounded h.  The scale is correctly rounded, and a
 * quotient half-way between two e4m3 values goes to the even one.
 *   dtype         a quant_type_t: the type of x, residual, weight,
 *                 residual_out and y
 *   residual      may be NULL; residual_out, y, and q with scale may be NULL
 *                 (not computed), but not all of them.  q and scale go
 *                 together (cols = 0: scale alone).
 *   residual_out  may be the same buffer as x or residual (same leading
 *                 dimension); so may y
 *   eps           >= 0
 * No alignment is asked for beyond the element's own; rows on 16-byte
 * boundaries (8-byte for q) are the fast case.  A NaN or an infinity in a row
 * of h or of y makes that row's q and scale NaN, and y what the formula gives
 * (a row of zeros with eps = 0: NaN).  A row whose squares, or their sum, leave
 * fp32's range is scaled by a power of two first: every finite h has its y.
 * cols = 0 writes scale alone, 2^-126 a row.
 */
int add_rmsnorm(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual,
                int64_t ldr, const void* weight, float eps, int dtype, void* residual_out,
                int64_t ldro, void* y, int64_t ldy, void* q, int64_t ldq, float* scale,
                void* stream);

/*
 * quantize_fp8 -- scale = max(max|x| / 448, 2^-126) and q = e4m3(x / scale)
 * for each row: activations without a norm, or a weight matrix stored N x K
 * (a scale an output column).  A NaN or an infinity in a row of x makes that
 * row's q and scale NaN.  Types and alignment as add_rmsnorm.
 */
int quantize_fp8(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, void* q,
                 int64_t ldq, float* scale, void* stream);

/*
 * gemm_fp8 -- C[i,j] = a_scale[i] * b_scale[j] * sum_k A[i,k] * B[k,j]
 *   A        M x K e4m3, row-major, lda >= K
 *   B        K x N e4m3, column-major: element (k,j) at B[j*ldb + k], ldb >= K
 *   C        M x N, row-major, ldc >= N; dtype QUANT_F16 or QUANT_BF16 (the
 *            fp32 result rounded to nearest even; fp16 overflows to infinity).
 *            QUANT_F32 is GEMM_ERR_UNSUPPORTED.
 *   a_scale, b_scale   M and N fp32 values
 * Products are summed in fp32 on the tensor cores; the sum is multiplied in fp32
 * by a_scale[i], then by b_scale[j].  K = 0 gives C = 0.
 * Alignment (GEMM_ERR_ALIGN otherwise): A, B and C start on 16-byte
 * boundaries and lda, ldb and ldc*2 are multiples of 16; a_scale and b_scale
 * are 4-byte aligned.
 */
int gemm_fp8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
             int64_t ldb, void* C, int64_t ldc, const float* a_scale, const float* b_scale,
             int dtype, void* stream);

/*
 * gemm_fp8_checked -- gemm_fp8, then synchronise `stream` and read (and clear)
 * the kernels' device status word: GEMM_ERR_TIMEOUT if a pipeline wait ran out
 * (C is then undefined; gemm_debug_set's hooks apply), GEMM_ERR_CUDA if the
 * stream reported an error.  Meant for tests and debugging.
 */
int gemm_fp8_checked(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                     int64_t ldb, void* C, int64_t ldc, const float* a_scale, const float* b_scale,
                     int dtype, void* stream);

/*
 * gemm_fp8_plan -- the launch gemm_fp8 would make for these sizes and this
 * dtype of C, without making it.  Needs a current CUDA device (it asks the
 * runtime how many clusters can be resident).  GEMM_ERR_ARG for sizes below 1,
 * an unknown dtype or a NULL plan; GEMM_ERR_UNSUPPORTED as gemm_fp8.
 */
int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int dtype, quant_plan_t* plan);

/*
 * gemv_w4 -- C[i,j] = sum_k x[i,k] * scales[j,k/group] * (w[j,k] - zeros[j,k/group])
 *   x        M x K, dtype QUANT_F16 or QUANT_BF16, ldx >= K
 *   W        N x K 4-bit values 0..15, two a byte, the even k in the low four
 *            bits: w[j,k] in byte W[j*ldw + k/2]; ldw >= K/2 bytes
 *   scales   N x K/group of x's type, lds >= K/group
 *   zeros    N x K/group bytes 0..15, ldz >= K/group; NULL: every zero point is 8
 *   group    32, 64 or 128; K is a multiple of it (GEMM_ERR_ARG otherwise)
 *   C        M x N of x's type, ldc >= N
 * Made for few rows: the weights are read once for every 16 or 32 rows of x.
 * Sums are fp32.  K = 0 gives C = 0.  A NaN or an infinity in x stays in its
 * row of C and acts as the formula says; one in scales stays in its column.
 * Alignment (GEMM_ERR_ALIGN otherwise): x and W start on 16-byte boundaries,
 * ldx*2 and ldw are multiples of 16; the others are aligned to their element.
 * K above 2^26 and lds or ldz above 2^22 are GEMM_ERR_UNSUPPORTED.
 */
int gemv_w4(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
            int64_t ldw, const void* scales, int64_t lds, const void* zeros, int64_t ldz,
            int group, void* C, int64_t ldc, int dtype, void* stream);

/* gemv_w4_checked -- gemv_w4 as gemm_fp8_checked is gemm_fp8. */
int gemv_w4_checked(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* W,
                    int64_t ldw, const void* scales, int64_t lds, const void* zeros, int64_t ldz,
                    int group, void* C, int64_t ldc, int dtype, void* stream);

/* gemv_w4_plan -- for gemv_w4 what gemm_fp8_plan is for gemm_fp8; `zeros` says
 * whether there are zero points (0 or 1). */
int gemv_w4_plan(int64_t M, int64_t N, int64_t K, int group, int zeros, int dtype, quant_plan_t* plan);

/*
 * quantize_w4 -- a weight matrix (N x K, row-major, any quant_type_t) in the
 * form gemv_w4 reads, with scales of `scale_dtype` (QUANT_F16 or QUANT_BF16).
 * A group's scale is max|w|/7 with zero point 8 (zeros = NULL), or
 * (max(w,0) - min(w,0))/15 with zero point round(-min(w,0)/scale), limited to
 * 15; it is rounded to scale_dtype first (to its largest finite value at most),
 * and w is then round(w/scale) + zero point, limited to 0..15, round to nearest
 * even and round(w/0) = 0.  Weights are finite.  Arguments otherwise as gemv_w4; no
 * alignment beyond the elements' own, and ldw need only be >= K/2.
 */
int quantize_w4(int64_t N, int64_t K, const void* w, int64_t ld, int dtype, int group, void* W,
                int64_t ldw, void* scales, int64_t lds, int scale_dtype, void* zeros, int64_t ldz,
                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSP_QUANT_H */
