// orthogonalize.cu -- Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T,
// on the tensor cores, and the two passes before them: the sum of squares, and
// the first X.
//
// A step is three products (product_*_sm103a.cu).  The first two are symmetric,
// so where a matrix has many tiles only those on and below the diagonal are
// computed and mirrored.  The polynomial's coefficients are epilogue factors:
// nothing but X, A and b A + c A^2 is ever written.  A tall matrix is not
// transposed: A = X^T X takes both operands MN-major.
//
// Between the products everything is fp16 at power-of-two scales, which cost
// nothing (they go into the same factors) and put the elements where fp16 has
// all its 11 bits: X of spectral norm one has elements about 1 / sqrt(longer
// side), A about 1 / shorter side off its diagonal.  bf16 would lose three of
// those bits for a range that is not needed.  The first X is G times a power of
// two, exact for 16-bit gradients whose elements lie within fp16's range of one
// another; what is left of the norm, t, is applied to the first step's factors,
// on the device.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "linear.h"
#include "ortho.cuh"

namespace ssp {
namespace {

constexpr int THREADS = 256;
constexpr int kMostParts = 1024;  // CTAs that share a matrix's sum
constexpr int AHEAD = 4;          // groups of eight a thread has under way

struct Params {
    int rows, cols;
    int vecs;  // groups of eight elements a row
    // Row of group i: i * by >> shift, exact for i < 2^27 (a division otherwise
    // takes longer than the group).
    uint32_t by;
    int shift;
    OrthoInput in;
    double* parts;  // [batch][gridDim.x]: sums of squares
    int n_parts;
    float eps;
    int exponent;  // of the first X's norm
    // What the second pass writes: the first X, or (no steps) the output.
    void* out;
    long long ldo, stride_o;
    int out_bf16, last;
    float scale;
    float* factor;
};

struct Place {
    int row, col;
};
__device__ __forceinline__ Place place_of(const Params& p, int i) {
    const int row = static_cast<int>(static_cast<uint64_t>(i) * p.by >> p.shift);
    return {row, (i - row * p.vecs) * 8};
}

// f(place, values) for this thread's share of matrix b's groups of eight.
template <int TYPE, class F>
__device__ __forceinline__ void each_group(const Params& p, int b, F&& f) {
    const int n = p.rows * p.vecs, stride = static_cast<int>(gridDim.x) * THREADS;
    for (int i = static_cast<int>(blockIdx.x) * THREADS + static_cast<int>(threadIdx.x); i < n; i += AHEAD * stride) {
        Place at[AHEAD];
        Raw raw[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i + k * stride < n) {
                at[k] = place_of(p, i + k * stride);
                raw[k] = load_raw<TYPE>(p.in, b, at[k].row, at[k].col, p.cols - at[k].col);
            }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i + k * stride < n) {
                float v[8];
                values<TYPE>(raw[k], v);
                f(at[k], v);
            }
    }
}

template <int TYPE>
__global__ void __launch_bounds__(THREADS) ortho_sum_kernel(const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    const int b = static_cast<int>(blockIdx.y);
    SquareSum sq;
    each_group<TYPE>(p, b, [&](Place, const float(&v)[8]) { sq.add(v); });
    __shared__ double warps[THREADS / 32];
    const double mine = sq.warp_total();
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < THREADS / 32; ++w) s += warps[w];
        p.parts[static_cast<long long>(b) * gridDim.x + blockIdx.x] = s;
    }
}

// The first X, G 2^e, or (no steps) the output.
template <int TYPE>
__global__ void __launch_bounds__(THREADS) ortho_first_kernel(const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    const int b = static_cast<int>(blockIdx.y);
    __shared__ float factors[3];
    if (threadIdx.x < 32) {
        double v = 0.0;
        for (int i = static_cast<int>(threadIdx.x); i < p.n_parts; i += 32)
            v += p.parts[static_cast<long long>(b) * p.n_parts + i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (threadIdx.x == 0) {
            first_factors(v, p.exponent, p.eps, factors);
            if (blockIdx.x == 0) p.factor[b] = factors[2];
        }
    }
    __syncthreads();
    const float by0 = factors[0], by1 = factors[1], after = p.last ? factors[2] * p.scale : 1.0f;
    each_group<TYPE>(p, b, [&](Place at, const float(&x)[8]) {
        const int c = at.col;
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            u[k] = pack16(p.out_bf16 != 0, x[2 * k] * by0 * by1 * after, x[2 * k + 1] * by0 * by1 * after);
        uint16_t* d = static_cast<uint16_t*>(p.out) + static_cast<long long>(b) * p.stride_o +
                      static_cast<long long>(at.row) * p.ldo + c;
        if (p.cols - c >= 8 || !p.last) {  // the first X's rows are padded to whole groups
            *reinterpret_cast<uint4*>(d) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < p.cols - c) d[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1)));
        }
    });
}

template <int TYPE>
int launch_first(const Params& p, int64_t batch, cudaStream_t stream) {
    ProductConfig c(1, 1, THREADS, 0, stream);
    c.cfg.gridDim = dim3(static_cast<unsigned>(p.n_parts), static_cast<unsigned>(batch));
    const int st = product_finish(cudaLaunchKernelEx(&c.cfg, ortho_sum_kernel<TYPE>, p));
    return st != GEMM_OK ? st : product_finish(cudaLaunchKernelEx(&c.cfg, ortho_first_kernel<TYPE>, p));
}

// Row length of a tensor in the workspace: whole 16 bytes for the tensor copies;
// whole 128-byte lines where that adds a quarter at most, so that no row of a copied
// box lies in two (two of 2528 x 7457 1170 us, with whole 16 bytes 1343).
int64_t padded(int64_t n) { return n < 256 ? (n + 7) / 8 * 8 : (n + 63) / 64 * 64; }

// Where the workspace's parts begin.
struct Layout {
    size_t factor, parts, x[2], a, b, bytes;
};
Layout layout(int64_t batch, int64_t rows, int64_t cols) {
    const int64_t n = rows < cols ? rows : cols;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += (bytes + 255) / 256 * 256;
        return r;
    };
    Layout l;
    const size_t k = static_cast<size_t>(batch);
    l.factor = take(k * sizeof(float));
    l.parts = take(k * kMostParts * sizeof(double));
    for (size_t& x : l.x) x = take(k * rows * padded(cols) * 2);
    l.a = take(k * n * padded(n) * 2);
    l.b = take(k * n * padded(n) * 2);
    l.bytes = at;
    return l;
}

}  // namespace

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols) { return layout(batch, rows, cols).bytes; }

int ortho_launch(const OrthoLaunch& L, cudaStream_t stream) {
    if (ortho_small_takes(L)) return ortho_small_launch(L, stream);
    const Layout at = layout(L.batch, L.rows, L.cols);
    uint8_t* ws = static_cast<uint8_t*>(L.workspace);
    const bool tall = L.rows > L.cols;
    const int64_t n = tall ? L.cols : L.rows, m = tall ? L.rows : L.cols;
    Params p = {};
    p.rows = static_cast<int>(L.rows);
    p.cols = static_cast<int>(L.cols);
    p.vecs = static_cast<int>((L.cols + 7) / 8);
    p.in = {L.g, L.ldg, L.stride_g};
    p.parts = reinterpret_cast<double*>(ws + at.parts);
    int bits = 0;
    while ((1 << bits) < p.vecs) ++bits;
    p.shift = 27 + bits;
    p.by = static_cast<uint32_t>(((uint64_t{1} << p.shift) + p.vecs - 1) / p.vecs);
    // AHEAD groups a thread before another CTA takes part, eight CTAs an SM at most.
    const int64_t groups = static_cast<int64_t>(p.rows) * p.vecs;
    const int64_t share = (groups + AHEAD * THREADS - 1) / (AHEAD * THREADS);
    const int64_t most = (kMostParts + L.batch - 1) / L.batch;
    p.n_parts = static_cast<int>(share < most ? share : most);
    p.eps = L.eps;
    const OrthoScales scales = ortho_scales(L.rows, L.cols);
    p.exponent = scales.exponent;
    p.scale = L.scale;
    p.factor = reinterpret_cast<float*>(ws + at.factor);
    p.last = L.steps == 0;
    const int64_t ldx = padded(L.cols), ldn = padded(n);
    if (p.last) {
        p.out = L.out;
        p.ldo = L.ldo;
        p.stride_o = L.stride_o;
        p.out_bf16 = L.out_bf16;
    } else {
        p.out = ws + at.x[0];
        p.ldo = ldx;
        p.stride_o = L.rows * ldx;
    }
    int st = L.dtype == QUANT_F32    ? launch_first<QUANT_F32>(p, L.batch, stream)
             : L.dtype == QUANT_BF16 ? launch_first<QUANT_BF16>(p, L.batch, stream)
                                     : launch_first<QUANT_F16>(p, L.batch, stream);
    const double sa = scales.a, sx = scales.x;
    for (int s = 0; st == GEMM_OK && s < L.steps; ++s) {
        const bool first = s == 0, last = s + 1 == L.steps;
        const ProductMatrix X = {ws + at.x[s & 1], ldx, L.rows * ldx};
        const ProductMatrix A = {ws + at.a, ldn, n * ldn}, B = {ws + at.b, ldn, n * ldn};
        ProductLaunch q;
        q.batch = L.batch;
        q.epi = EPI_STEP;
        q.padded = 1;
        q.factor = p.factor;
        // A = X X^T, or X^T X
        q.M = q.N = n;
        q.K = m;
        q.A = q.B = X;
        q.a_mn = q.b_mn = tall;
        q.symmetric = 1;
        q.D = A;
        q.alpha = static_cast<float>(first ? sa : sa / (sx * sx));
        q.alpha_pow = first ? 2 : 0;
        if ((st = product_launch(q, stream)) != GEMM_OK) break;
        // B = b A + c A^2
        q.K = n;
        q.A = q.B = q.R = A;
        q.a_mn = q.b_mn = 0;
        q.D = B;
        q.alpha = static_cast<float>(L.c / sa);
        q.alpha_pow = 0;
        q.beta = L.b;
        if ((st = product_launch(q, stream)) != GEMM_OK) break;
        // X = a X + B X, or a X + X B
        const double sn = last ? static_cast<double>(L.scale) : sx;  // what the new X is multiplied by
        q.M = L.rows;
        q.N = L.cols;
        q.A = tall ? X : B;
        q.B = tall ? B : X;
        q.b_mn = !tall;
        q.symmetric = 0;
        q.R = X;
        q.alpha = static_cast<float>(first ? sn / sa : sn / (sa * sx));
        q.beta = static_cast<float>(first ? L.a * sn : L.a * sn / sx);
        q.alpha_pow = q.beta_pow = first;
        if (last) {
            q.padded = 0;
            q.D = {L.out, L.ldo, L.stride_o};
            q.out_bf16 = L.out_bf16;
        } else {
            q.D = {ws + at.x[(s + 1) & 1], ldx, L.rows * ldx};
        }
        st = product_launch(q, stream);
    }
    return st;
}

}  // namespace ssp
