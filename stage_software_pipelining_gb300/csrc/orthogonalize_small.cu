// orthogonalize_small.cu -- all Newton-Schulz steps of matrices with a side of 128
// at most in one launch.
//
// As three products a step (orthogonalize.cu) such a matrix takes 17 launches of
// some 4 us, whatever its size.  Here a cluster of CTAs holds X in shared memory for
// all steps, each a slice of the longer side, and a step is
//
//     A = X X^T     every CTA over its slice (tcgen05), the partials joined through
//                   distributed shared memory, in rank order
//     B = b A + c A^2     by every CTA for itself: 128^3 is no work
//     X = a X + B X       every CTA its slice
//
// X's fp16 slice lies in blocks of 64 columns, 128 rows of a 128-byte
// swizzle row each: read as a K-major operand it is X for A, read as an MN-major
// operand it is X for B X, so it is never rearranged.  A, b A + c A^2 and X are
// rounded where orthogonalize.cu rounds them, at the same scales.
//
// Bound by latencies, some 1.2 us a product and 4 us a step for the cluster's
// exchange: in a graph 128 x 128 takes 22.5 us (as products 54), 128 x 1024 46 (60).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "internal.h"
#include "ortho.cuh"
#include "product.cuh"

namespace ssp {

__device__ GemmDeviceStatus g_ortho_small_status;

namespace {

constexpr int THREADS = 256;
constexpr int SIDE = 128;             // rows of X held, zeros past the matrix's
constexpr int BLOCK = SIDE * 128;     // 64 columns of X, A or B
constexpr int kMostSlice = 320;       // columns of a CTA: what shared memory holds
constexpr int kMostCluster = 8;

struct Params {
    OrthoInput in;
    int n, m;     // X's rows (the shorter side) and columns
    int tall;     // X is the transpose
    int w;        // columns of a CTA's slice, a multiple of 64
    int steps;
    float a, b, c, eps, scale;
    int exponent;   // of the first X's norm
    float sa, sx;   // scales of A and B, and of X
    uint32_t idesc_a, idesc_x;  // 128 x 128, K-major; 128 x 64 with X MN-major (N to be set)
    void* out;
    long long ldo, stride_o;
    int out_bf16;
    unsigned long long wait_limit_ns;
    int withhold;
};

struct Ctl {
    unsigned long long bar, drain;
    int failed;       // a wait ran out
    double sum;       // of squares, this CTA's slice
    uint32_t tmem_base;
    float factors[3];
    double warps[THREADS / 32];
};

// Room for a cluster's partials: ceil(128 / split) rows of each CTA.
__host__ __device__ __forceinline__ int join_bytes(int split) {
    return split > 1 ? split * ((SIDE + split - 1) / split) * SIDE * 4 : 0;
}

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_u2(uint32_t cluster_addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(x), "r"(y) : "memory");
}

// Piece j (16 bytes) of row i of a block.
__device__ __forceinline__ uint32_t piece(uint32_t block, int i, int j) {
    return block + static_cast<uint32_t>(i) * 128u + static_cast<uint32_t>((j ^ (i & 7)) << 4);
}

template <int TYPE>
__global__ void __launch_bounds__(THREADS, 1) ortho_small_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t X = smem_addr(smem);
    const uint32_t A = X + static_cast<uint32_t>(p.w / 64) * BLOCK;  // two blocks
    const uint32_t B = A + 2 * BLOCK;                                // two blocks
    // What the cluster's CTAs have for this one's share of A's rows, fp32: [CTA][row
    // of the share][128], 16-byte pieces turned by the row.
    const uint32_t P = B + 2 * BLOCK;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + (p.w / 64 + 4) * BLOCK + join_bytes(static_cast<int>(gridDim.x)));

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int split = static_cast<int>(gridDim.x);  // a cluster is a row of the grid
    const int rank = static_cast<int>(blockIdx.x);
    const int b = static_cast<int>(blockIdx.y);
    const int j0 = rank * p.w;                      // the slice's first column
    const int cols = max(0, min(p.w, p.m - j0));    // those of the matrix
    const int most = (SIDE + split - 1) / split;    // rows of A that a CTA joins
    const uint32_t bar = smem_addr(&ctl->bar);

    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->failed = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&ctl->tmem_base), 512u);
        tmem_relinquish();
        tc_fence_before();
    }
    for (int i = tid; i < p.w / 64 * (BLOCK / 16); i += THREADS) st_shared_v4(X + 16u * i, make_uint4(0u, 0u, 0u, 0u));
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    griddep_wait();
    griddep_launch_dependents();

    // The slice in G: its rows [j0, j0 + cols) where X is the transpose, else those
    // columns; groups of eight elements of a row.
    const int g_rows = p.tall ? cols : p.n, g_cols = p.tall ? p.n : cols;
    const int vecs = (g_cols + 7) / 8, groups = vecs > 0 ? g_rows * vecs : 0;
    auto each = [&](auto f) {
        constexpr int AHEAD = 8;  // groups a thread has under way
        for (int i0 = tid; i0 < groups; i0 += AHEAD * THREADS) {
            Raw raw[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int i = min(i0 + k * THREADS, groups - 1), r = i / vecs, c = (i - r * vecs) * 8;
                // (a slice's last columns are followed by the next one's: they are
                // counted out)
                raw[k] = load_raw<TYPE>(p.in, b, p.tall ? j0 + r : r, p.tall ? c : j0 + c, g_cols - c);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int i = i0 + k * THREADS, r = i / vecs, c = (i - r * vecs) * 8;
                if (i < groups) {
                    float v[8];
                    values<TYPE>(raw[k], v);
                    f(r, c, v);
                }
            }
        }
    };
    SquareSum sq;
    each([&](int, int, const float(&v)[8]) { sq.add(v); });
    const double s = sq.warp_total();
    if (lane == 0) ctl->warps[warp] = s;
    __syncthreads();
    if (tid == 0) {
        double t = 0.0;
        for (int k = 0; k < THREADS / 32; ++k) t += ctl->warps[k];
        ctl->sum = t;
    }
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    if (tid == 0) {
        double total = 0.0;
        for (int r = 0; r < split; ++r) {
            const uint32_t at = mapa_shared(smem_addr(&ctl->sum), static_cast<uint32_t>(r));
            double t;
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(t) : "r"(at) : "memory");
            total += t;
        }
        first_factors(total, p.exponent, p.eps, ctl->factors);
    }
    __syncthreads();
    const float by0 = ctl->factors[0], by1 = ctl->factors[1], t = ctl->factors[2];
    each([&](int r, int c, const float(&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = pack16<false>(v[2 * k] * by0 * by1, v[2 * k + 1] * by0 * by1);
        if (!p.tall) {
            st_shared_v4(piece(X + static_cast<uint32_t>(c / 64) * BLOCK, r, c % 64 / 8), make_uint4(u[0], u[1], u[2], u[3]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < p.n)
                    st_shared_u16(piece(X + static_cast<uint32_t>(r / 64) * BLOCK, c + k, r % 64 / 8) + r % 8 * 2,
                                  static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1))));
        }
    });
    fence_proxy_async_shared();
    __syncthreads();

    // A wait that runs out ends this CTA's products and waits; it still takes part in
    // the barriers, and leaves when the products on their way have landed.  (Its threads
    // learn of it in their waits: a look at the flag beside each takes 0.06 us.)
    volatile int* failed = &ctl->failed;
    const int withhold = rank == 0 && b == 0 ? p.withhold : -1;
    uint32_t phase = 0;
    bool ok = true;
    // Waits until the products issued before the last commit are done.
    auto products_done = [&]() {
        if (ok && !mbar_try_wait(bar, phase)) {
            const unsigned long long t0 = globaltimer_ns();
            while (ok && !mbar_try_wait(bar, phase)) {
                if (*failed) {
                    ok = false;
                } else if (globaltimer_ns() - t0 > p.wait_limit_ns) {
                    record_product_timeout(&g_ortho_small_status, P_EPILOGUE, 0);
                    *failed = 1;
                    ok = false;
                }
            }
        }
        phase ^= 1u;
        tc_fence_after();
    };
    // The thread that issues the products: the commit of number n (three a step).
    auto commit = [&](int n) {
        if (n != withhold) umma_commit(bar);
    };
    const int q = warp & 3, half = warp >> 2;  // TMEM lanes 32q.., and which blocks of 64 columns
    const int i = 32 * q + lane;               // this thread's row
    const uint32_t t_row = tmem + (static_cast<uint32_t>(32 * q) << 16);
    // Thirty-two columns of this thread's row.  Every use is in a loop that is not
    // unrolled: the steps' code is to stay in the instruction cache.
    auto sums = [&](int col, uint32_t (&r)[32]) {
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(col), r);
        tmem_ld_wait();
    };
    for (int step = 0; step < p.steps; ++step) {
        const bool first = step == 0, last = step + 1 == p.steps;
        // ---- A = X X^T
        if (warp == 0 && elect_one_sync() && ok) {
            const uint64_t d = operand_desc(X, 0);
            for (int k = 0; k < p.w / 16; ++k) {
                const uint64_t at = d + static_cast<uint32_t>(k / 4 * (BLOCK / 16) + k % 4 * 2);
                umma_f16(tmem, at, at, p.idesc_a, k != 0);
            }
            commit(3 * step);
        }
        __syncwarp();
        products_done();
        const float alpha = first ? p.sa * t * t : p.sa / (p.sx * p.sx);
#pragma unroll 1
        for (int h = 2 * half; h < 2 * half + 2; ++h) {  // columns 32h..
            uint32_t r[32];
            sums(32 * h, r);
            if (split == 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        u[k] = pack16<false>(alpha * __uint_as_float(r[8 * j + 2 * k]), alpha * __uint_as_float(r[8 * j + 2 * k + 1]));
                    st_shared_v4(piece(A + static_cast<uint32_t>(half) * BLOCK, i, 4 * (h & 1) + j),
                                 make_uint4(u[0], u[1], u[2], u[3]));
                }
            } else {
                // Each CTA joins a share of the rows: it gets them from all.
                const int owner = ((i + 1) * split - 1) / SIDE;
                const uint32_t to = mapa_shared(P + static_cast<uint32_t>(rank * most + i - SIDE * owner / split) * 512u,
                                                static_cast<uint32_t>(owner));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_cluster_f4(to + static_cast<uint32_t>(((8 * h + j) ^ lane) << 4),
                                  make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                              __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
            }
        }
        tc_fence_before();
        if (split > 1) {
            cluster_sync_all();
            const int r0 = SIDE * rank / split, r1 = SIDE * (rank + 1) / split;
            for (int e = tid; e < (r1 - r0) * 32; e += THREADS) {
                const int row = r0 + e / 32, c4 = e % 32;
                const uint32_t at = P + static_cast<uint32_t>(e / 32) * 512u + static_cast<uint32_t>((c4 ^ (row & 31)) << 4);
                float4 v = {};
#pragma unroll 4
                for (int r = 0; r < split; ++r) {
                    const uint4 u = ld_shared_v4(at + static_cast<uint32_t>(r * most) * 512u);
                    v = make_float4(v.x + __uint_as_float(u.x), v.y + __uint_as_float(u.y), v.z + __uint_as_float(u.z),
                                    v.w + __uint_as_float(u.w));
                }
                // ... and hands it to all.
                const uint32_t to = piece(A + static_cast<uint32_t>(c4 / 16) * BLOCK, row, c4 % 16 / 2) + c4 % 2 * 8;
                const uint32_t lo = pack16<false>(alpha * v.x, alpha * v.y), hi = pack16<false>(alpha * v.z, alpha * v.w);
                for (int r = 0; r < split; ++r) st_cluster_u2(mapa_shared(to, static_cast<uint32_t>(r)), lo, hi);
            }
            fence_proxy_async_all();
            cluster_sync_all();
        }
        fence_proxy_async_all();
        __syncthreads();
        tc_fence_after();
        // ---- B = b A + c A^2
        if (warp == 0 && elect_one_sync() && ok) {
            const uint64_t d = operand_desc(A, 0);
#pragma unroll
            for (int k = 0; k < SIDE / 16; ++k) {
                const uint64_t at = d + static_cast<uint32_t>(k / 4 * (BLOCK / 16) + k % 4 * 2);
                umma_f16(tmem, at, at, p.idesc_a, k != 0);
            }
            commit(3 * step + 1);
        }
        __syncwarp();
        products_done();
        const float gamma = p.c / p.sa;
#pragma unroll 1
        for (int h = 2 * half; h < 2 * half + 2; ++h) {
            uint32_t r[32];
            sums(32 * h, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 old = ld_shared_v4(piece(A + static_cast<uint32_t>(half) * BLOCK, i, 4 * (h & 1) + j));
                const uint32_t w[4] = {old.x, old.y, old.z, old.w};
                uint32_t u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack16<false>(w[k]);
                    u[k] = pack16<false>(fmaf(p.b, f.x, gamma * __uint_as_float(r[8 * j + 2 * k])),
                                         fmaf(p.b, f.y, gamma * __uint_as_float(r[8 * j + 2 * k + 1])));
                }
                st_shared_v4(piece(B + static_cast<uint32_t>(half) * BLOCK, i, 4 * (h & 1) + j),
                             make_uint4(u[0], u[1], u[2], u[3]));
            }
        }
        tc_fence_before();
        fence_proxy_async_shared();
        __syncthreads();
        tc_fence_after();
        // ---- X = a X + B X
        if (warp == 0 && elect_one_sync() && ok) {
            const uint64_t db = operand_desc(B, 0);
            // X as an MN-major operand: blocks of 64 columns are BLOCK bytes apart.
            const uint64_t dx = (operand_desc(X, 1) & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(BLOCK / 16) << 16);
            for (int c = 0; c < p.w; c += 256) {
                const uint32_t wide = static_cast<uint32_t>(min(256, p.w - c));
                const uint32_t idesc = p.idesc_x | ((wide >> 3) << 17);
#pragma unroll
                for (int k = 0; k < SIDE / 16; ++k)
                    umma_f16(tmem + static_cast<uint32_t>(c), db + static_cast<uint32_t>(k / 4 * (BLOCK / 16) + k % 4 * 2),
                             dx + static_cast<uint32_t>(c / 64 * (BLOCK / 16) + k * (2048 / 16)), idesc, k != 0);
            }
            commit(3 * step + 2);
        }
        __syncwarp();
        products_done();
        const float sn = last ? p.scale : p.sx;  // what the new X is multiplied by
        const float by_sum = first ? sn / p.sa * t : sn / (p.sa * p.sx), by_old = first ? p.a * sn * t : p.a * sn / p.sx;
        uint16_t* const o = static_cast<uint16_t*>(p.out) + b * p.stride_o;
#pragma unroll 1
        for (int h = half; h < p.w / 32; h += 2) {  // columns 32h.. of the slice
            uint32_t r[32];
            sums(32 * h, r);
            const uint32_t xb = X + static_cast<uint32_t>(h / 2) * BLOCK;
#pragma unroll
            for (int k8 = 0; k8 < 4; ++k8) {
                const uint32_t at = piece(xb, i, 4 * (h & 1) + k8);
                const uint4 old = ld_shared_v4(at);
                const uint32_t w[4] = {old.x, old.y, old.z, old.w};
                uint32_t u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack16<false>(w[k]);
                    u[k] = pack16(last && p.out_bf16, fmaf(by_old, f.x, by_sum * __uint_as_float(r[8 * k8 + 2 * k])),
                                  fmaf(by_old, f.y, by_sum * __uint_as_float(r[8 * k8 + 2 * k + 1])));
                }
                // (the output, too, leaves by way of X's place)
                st_shared_v4(at, make_uint4(u[0], u[1], u[2], u[3]));
            }
        }
        if (last) {
            __syncthreads();
            if (!p.tall) {
                // Eight columns of a row a thread.
                for (int e = tid; e < p.n * (p.w / 8); e += THREADS) {
                    const int row = e / (p.w / 8), c = e % (p.w / 8) * 8, left = cols - c;
                    const uint4 v = ld_shared_v4(piece(X + static_cast<uint32_t>(c / 64) * BLOCK, row, c % 64 / 8));
                    uint16_t* d = o + row * p.ldo + j0 + c;
                    if (left >= 8) {
                        *reinterpret_cast<uint4*>(d) = v;
                    } else {
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 7; ++k)
                            if (k < left) d[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1)));
                    }
                }
            } else {
                // A row of the output is a column of X: adjacent lanes, adjacent rows of X.
                const uint8_t* x = smem;
                for (int e = tid; e < cols * SIDE; e += THREADS) {
                    const int row = e % SIDE, c = e / SIDE;
                    if (row < p.n)
                        o[(j0 + c) * p.ldo + row] = *reinterpret_cast<const uint16_t*>(
                            x + (piece(X + static_cast<uint32_t>(c / 64) * BLOCK, row, c % 64 / 8) - X) + c % 8 * 2);
                }
            }
            break;
        }
        tc_fence_before();
        fence_proxy_async_shared();
        __syncthreads();
        tc_fence_after();
    }
    if (*failed) {  // (set before the last barrier)
        if (warp == 0) {
            const uint32_t drain = smem_addr(&ctl->drain);
            if (elect_one_sync()) umma_commit(drain);
            __syncwarp();
            drain_wait(drain, 0u, p.wait_limit_ns);
        }
        __syncthreads();
    }
    if (split > 1) cluster_sync_all();  // no CTA leaves while another reads its shared memory
    if (warp == 1) tmem_dealloc(tmem, 512u);
}

template <int TYPE>
int launch(const Params& p, int split, int64_t batch, cudaStream_t stream) {
    static std::mutex mu;
    static bool done[64] = {};
    auto kernel = ortho_small_kernel<TYPE>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GEMM_ERR_CUDA;
    {
        std::lock_guard<std::mutex> g(mu);
        if (!done[dev])
            done[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem) == cudaSuccess;
        if (!done[dev]) return GEMM_ERR_LAUNCH;
    }
    size_t smem = 1024 + static_cast<size_t>(p.w / 64 + 4) * BLOCK + join_bytes(split) + sizeof(Ctl);
    static_assert(1024 + (kMostSlice / 64 + 4) * BLOCK + (SIDE + kMostCluster) * SIDE * 4 + sizeof(Ctl) <= kProductSmem,
                  "shared memory");
    if (smem < kTmemAloneSmem) smem = kTmemAloneSmem;
    ProductConfig c(split, split, THREADS, smem, stream);
    c.cfg.gridDim = dim3(static_cast<unsigned>(split), static_cast<unsigned>(batch));
    return product_finish(cudaLaunchKernelEx(&c.cfg, kernel, p));
}

}  // namespace

bool ortho_small_takes(const OrthoLaunch& L) {
    const int64_t n = L.rows < L.cols ? L.rows : L.cols, m = L.rows < L.cols ? L.cols : L.rows;
    return L.steps > 0 && n <= SIDE && m <= kMostSlice * kMostCluster;
}

int ortho_small_launch(const OrthoLaunch& L, cudaStream_t stream) {
    Params p = {};
    p.tall = L.rows > L.cols;
    p.n = static_cast<int>(p.tall ? L.cols : L.rows);
    p.m = static_cast<int>(p.tall ? L.rows : L.cols);
    p.in = {L.g, L.ldg, L.stride_g};
    p.steps = L.steps;
    p.a = L.a;
    p.b = L.b;
    p.c = L.c;
    p.eps = L.eps;
    p.scale = L.scale;
    const OrthoScales s = ortho_scales(L.rows, L.cols);
    p.exponent = s.exponent;
    p.sa = s.a;
    p.sx = s.x;
    p.out = L.out;
    p.ldo = L.ldo;
    p.stride_o = L.stride_o;
    p.out_bf16 = L.out_bf16;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    // The slice's width with the least time: rounds of clusters that run at once, each
    // the steps' latency, the slice's work and, in a cluster, the exchange.  (us;
    // measured: 128 x 128 in one CTA 22.6, 128 x 1024 in eight of 128 columns 46, in four
    // of 256 53, 100 x 304 in one of 320 34, in three of 128 42.)
    int resident[9];
    if (!product_resident_ctas(resident)) return GEMM_ERR_CUDA;
    double least = 1e30;
    for (int w = 64; w <= kMostSlice; w += 64) {
        const int c = (p.m + w - 1) / w;
        if (c > kMostCluster || resident[c] < c) continue;
        const int64_t at_once = resident[c] / c, rounds = (L.batch + at_once - 1) / at_once;
        const double us = static_cast<double>(rounds) * (3.0 + p.steps * (3.5 + 0.0145 * (w - 64) + (c > 1 ? 4.2 : 0.0)));
        if (us < least) {
            least = us;
            p.w = w;
        }
    }
    if (p.w == 0) return GEMM_ERR_LAUNCH;
    p.idesc_a = product_instruction(128, 128, 0, 0, 0);
    p.idesc_x = product_instruction(128, 0, 0, 0, 1);
    const int split = (p.m + p.w - 1) / p.w;
    return L.dtype == QUANT_F32    ? launch<QUANT_F32>(p, split, L.batch, stream)
           : L.dtype == QUANT_BF16 ? launch<QUANT_BF16>(p, split, L.batch, stream)
                                   : launch<QUANT_F16>(p, split, L.batch, stream);
}

int ortho_small_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_ortho_small_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_ortho_small_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
