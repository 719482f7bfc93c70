// gemm_fp8_sm103a.cu -- C[i,j] = a_scale[i] * b_scale[j] * sum_k A[i,k] B[k,j]
// with e4m3 A (row-major) and B (column-major: the N x K weights) and a
// 16-bit C, on the fifth-generation tensor cores.
//
// The scales do not depend on k, so the mainloop is a plain e4m3 product with
// fp32 accumulation in TMEM (tcgen05.mma kind::f8f6f4, K = 32 a step) and the
// epilogue multiplies by both.  A stage of the operand ring is one 128-byte
// swizzle row of each operand, K = 128.
//
// Two kernels:
//   * fp8_pair_kernel, many rows: 256 x 256 tiles of C on CTA pairs
//     (cta_group::2), persistent, two accumulators in TMEM so that a tile's
//     epilogue runs under the next tile's mainloop.  Bound by the tensor pipe.
//   * fp8_few_kernel, few rows: the roles of the operands are exchanged.  128
//     weight rows are the MMA's M side and the MT <= 256 rows of A its N
//     side, so one row of A costs a 16-wide MMA instead of a 128-row tile that
//     is empty but for one row.  K is cut over the CTAs of a cluster, whose
//     fp32 partials meet in distributed shared memory, so that a narrow
//     product still keeps every SM loading.  Bound by reading the weights.
//
// Every wait is bounded (gemm_debug_set's limit, 2 s unless set): a wait that
// runs out records the failure, raises the CTA's abort flag, lets the copies
// and MMAs in flight land and ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "../../include/quant.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant.h"

namespace ssp {

__device__ GemmDeviceStatus g_fp8_status;

namespace {

constexpr int BK = 128;                 // K of a stage: one 128-byte swizzle row of 8-bit values
constexpr int UMMA_K = 32;              // K per tcgen05.mma (kind::f8f6f4)
constexpr int ROW_TILE_BYTES = 128 * BK;  // 128 rows of a stage: 16 KB
constexpr int NUM_THREADS = 192;        // TMA warp, MMA warp, four epilogue warps
constexpr int kMaxSmem = 227 * 1024;
constexpr int kPairStages = 6;
constexpr int kPairBoxes = 2;           // output boxes per epilogue warp
constexpr int EPI_BOX_BYTES = 4096;     // 32 rows x 128 bytes
constexpr int ROLE_PRODUCER = 0, ROLE_MMA = 1, ROLE_EPILOGUE = 2;

struct Fp8Params {
    int M, N, K;
    int tiles_m, tiles_n, k_blocks;
    int group_m;   // pair kernel: tile rows walked together
    int split;     // few-row kernel: CTAs of a cluster, each with a part of K
    int stages;
    uint32_t idesc;
    int out_bf16;
    void* C;
    long long ldc;
    const float* a_scale;
    const float* b_scale;
    unsigned long long wait_limit_ns;
    int withhold;
};

// Shared-memory matrix descriptor of a K-major operand: 128-byte rows, 8-row
// groups 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void record_timeout(int role, int iter) {
    if (atomicCAS(&g_fp8_status.code, 0, GEMM_ERR_TIMEOUT) == 0) {
        g_fp8_status.block = blockIdx.x;
        g_fp8_status.role = role;
        g_fp8_status.iter = iter;
        __threadfence();
    }
}

// Wait for the phase of `bar` with parity `parity`; false after limit_ns or
// once another role has raised the abort flag.  PAIR: the peer CTA's flag is
// raised too.
template <bool PAIR>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                             unsigned long long limit_ns, int role, int iter) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                record_timeout(role, iter);
                *abort = 1;
                if constexpr (PAIR)
                    st_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(abort)),
                                               (cluster_ctarank() & 1u) ^ 1u),
                                   1u);
                return false;
            }
        }
    }
}

// After an abort: no flag check, still bounded.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity,
                                           unsigned long long limit_ns) {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) return;
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------- many rows
struct PairCtl {
    unsigned long long bar[2 * kPairStages + 5];  // full, empty, tmem_full[2], tmem_empty[2], drain
    uint32_t tmem_base;
    int abort;
    int epi_ok[2];  // the epilogue's go/abort decision, by tile parity
    alignas(16) float b_scale[256];
};

// Output tile of persistent work item t: groups of group_m tile rows walked
// column by column, every other group backwards, so that the pairs running
// at one time share A rows and weight rows in L2.
__device__ __forceinline__ void tile_coords(const Fp8Params& p, int t, int& tm, int& tn) {
    const int per_group = p.group_m * p.tiles_n;
    const int g = t / per_group;
    const int first_m = g * p.group_m;
    const int gsize = min(p.tiles_m - first_m, p.group_m);
    const int r = t - g * per_group;
    tm = first_m + r % gsize;
    tn = r / gsize;
    if (g & 1) tn = p.tiles_n - 1 - tn;
}

__device__ __forceinline__ void epilogue_bar_sync() { asm volatile("barrier.sync 1, 128;" ::: "memory"); }

// A cluster of two CTAs computes a 256 x 256 tile.  CTA rank r stages rows
// 128r.. of the A tile and weight rows 128r.. of the B tile; both CTAs' copies
// of a stage complete on the leader's full[s]; the leader issues every MMA and
// its commits free the stage in both CTAs.  Each CTA's TMEM receives its own
// 128 rows of C.
__global__ void __launch_bounds__(NUM_THREADS, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int S = kPairStages;
    uint8_t* a_ring = smem;
    uint8_t* b_ring = smem + S * ROW_TILE_BYTES;
    uint8_t* epi_ring = b_ring + S * ROW_TILE_BYTES;
    PairCtl* ctl = reinterpret_cast<PairCtl*>(epi_ring + 4 * kPairBoxes * EPI_BOX_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1u;
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
    const int tiles = p.tiles_m * p.tiles_n;
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
    volatile int* abort_flag = &ctl->abort;
    constexpr uint16_t kPairMask = 0x3;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmC);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 8);  // one arrive per epilogue warp of both CTAs
        }
        mbar_init(drain_bar, 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), 512u);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync_all();  // the peer's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    griddep_launch_dependents();
    griddep_wait();

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t leader_full0 = mapa_shared(full_bar(0), 0u);
            const uint64_t a_policy = l2_policy_evict_last();  // A rows serve the whole group of columns
            int s = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = unit; ok && t < tiles; t += units) {
                int tm, tn;
                tile_coords(p, t, tm, tn);
                const int a_row = tm * 256 + static_cast<int>(rank) * 128;
                const int b_row = tn * 256 + static_cast<int>(rank) * 128;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!bounded_wait<true>(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns,
                                            ROLE_PRODUCER, it)) {
                        ok = false;
                        break;
                    }
                    if (!(it == p.withhold && blockIdx.x == 0)) {
                        const uint32_t bar = leader_full0 + 8u * s;
                        if (leader) mbar_arrive_expect_tx(full_bar(s), 4u * ROW_TILE_BYTES);
                        tma_load_2d_pair_hint(smem_addr(a_ring + s * ROW_TILE_BYTES), &tmA, bar, kb * BK,
                                              a_row, a_policy);
                        tma_load_2d_pair(smem_addr(b_ring + s * ROW_TILE_BYTES), &tmB, bar, kb * BK, b_row);
                    }
                    ++it;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                if (leader) {
                    // Every copy this pair armed lands before the CTA exits.
                    for (int j = it - S > 0 ? it - S : 0; j < it; ++j) {
                        if (j == p.withhold && blockIdx.x == 0) continue;
                        drain_wait(full_bar(j % S), static_cast<uint32_t>((j / S) & 1), p.wait_limit_ns);
                    }
                } else {
                    // The peer's copies complete on the leader's barriers: a
                    // bounded grace period, then the closing cluster barrier
                    // keeps this CTA alive until the leader has drained.
                    const unsigned long long grace =
                        p.wait_limit_ns < 200000ull ? p.wait_limit_ns : 200000ull;
                    const unsigned long long t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < grace) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint64_t a_desc0 = smem_desc(smem_addr(a_ring));
            const uint64_t b_desc0 = smem_desc(smem_addr(b_ring));
            int s = 0, it = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto mma_wait = [&](uint32_t bar, uint32_t parity) -> bool {
                const bool r = bounded_wait<true>(bar, parity, abort_flag, p.wait_limit_ns, ROLE_MMA, it);
                return __all_sync(0xffffffffu, r) != 0;
            };
            for (int t = unit; ok && t < tiles; t += units, ++lt) {
                const int acc = lt & 1;
                if (!mma_wait(tempty_bar(acc), static_cast<uint32_t>((lt >> 1) & 1) ^ 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!mma_wait(full_bar(s), ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t off = static_cast<uint32_t>(s * ROW_TILE_BYTES) / 16u;
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                        if (elect_one_sync())
                            umma_f8_pair(d_tmem, a_desc0 + off + 2u * kk, b_desc0 + off + 2u * kk, p.idesc,
                                         (kb | kk) != 0);
                        __syncwarp();
                    }
                    if (elect_one_sync()) umma_commit_pair_multicast(empty_bar(s), kPairMask);
                    __syncwarp();
                    ++it;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if (elect_one_sync()) umma_commit_pair_multicast(tfull_bar(acc), kPairMask);
                __syncwarp();
            }
            if (!ok) {  // every MMA this warp issued finishes before TMEM is freed
                if (elect_one_sync()) umma_commit_pair_multicast(drain_bar, 0x1);
                __syncwarp();
                if (lane == 0) drain_wait(drain_bar, 0u, p.wait_limit_ns);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t tempty_leader0 = mapa_shared(tempty_bar(0), 0u);
        const uint32_t epi_buf0 = smem_addr(epi_ring) + static_cast<uint32_t>(q * kPairBoxes) * EPI_BOX_BYTES;
        const bool bf16 = p.out_bf16 != 0;
        const int et = (warp - 2) * 32 + lane;  // 0..127
        int lt = 0;
        uint32_t box = 0;  // boxes sent so far: their ring runs on from tile to tile
        for (int t = unit; t < tiles; t += units, ++lt) {
            const int acc = lt & 1;
            int tm, tn;
            tile_coords(p, t, tm, tn);
            const int row_base = tm * 256 + static_cast<int>(rank) * 128 + 32 * q;
            const int col0 = tn * 256;
            const float rs = row_base + lane < p.M ? p.a_scale[row_base + lane] : 0.0f;
            epilogue_bar_sync();  // the previous tile's column scales are read
            for (int c = et; c < 256; c += 128)
                ctl->b_scale[c] = col0 + c < p.N ? p.b_scale[col0 + c] : 0.0f;
            if (warp == 2 && lane == 0)
                ctl->epi_ok[lt & 1] = bounded_wait<true>(tfull_bar(acc), static_cast<uint32_t>((lt >> 1) & 1),
                                                         abort_flag, p.wait_limit_ns, ROLE_EPILOGUE, lt);
            __syncwarp();
            epilogue_bar_sync();
            if (!ctl->epi_ok[lt & 1]) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                   static_cast<uint32_t>(acc * 256);
            if (row_base < p.M) {
                const int boxes = min(4, (p.N - col0 + 63) / 64);
                for (int ci = 0; ci < boxes; ++ci) {
                    // Tensor stores clip rows past M, and columns past N in
                    // units of 16 bytes: a box with part of such a unit is
                    // written by each thread for its row.
                    const bool ragged = (p.N & 7) != 0 && col0 + ci * 64 + 64 > p.N;
                    const uint32_t buf = epi_buf0 + (box % kPairBoxes) * EPI_BOX_BYTES;
                    // The store that last used this box has read it.
                    if (lane == 0) bulk_wait_group_read<kPairBoxes - 1>();
                    __syncwarp();
                    uint32_t r[64];
                    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(ci * 64),
                                       *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
                    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(ci * 64 + 32),
                                       *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
                    tmem_ld_wait();
                    const float4* cs4 = reinterpret_cast<const float4*>(ctl->b_scale + ci * 64);
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj) {
                        const float4 c0 = cs4[2 * jj], c1 = cs4[2 * jj + 1];
                        const uint32_t* v = &r[8 * jj];
                        auto f = [&](int e, float cs) { return __uint_as_float(v[e]) * rs * cs; };
                        const uint4 u = make_uint4(pack16(f(0, c0.x), f(1, c0.y), bf16),
                                                   pack16(f(2, c0.z), f(3, c0.w), bf16),
                                                   pack16(f(4, c1.x), f(5, c1.y), bf16),
                                                   pack16(f(6, c1.z), f(7, c1.w), bf16));
                        if (!ragged) {
                            st_shared_v4(buf + lane * 128 + ((jj ^ (lane & 7)) << 4), u);
                        } else if (row_base + lane < p.M) {
                            const int n = col0 + ci * 64 + jj * 8;
                            uint16_t* c = static_cast<uint16_t*>(p.C) +
                                          static_cast<long long>(row_base + lane) * p.ldc + n;
                            if (n + 8 <= p.N) {
                                *reinterpret_cast<uint4*>(c) = u;
                            } else {
                                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (n + e < p.N) c[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                    if (ragged) continue;
                    ++box;
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tmC, buf, col0 + ci * 64, row_base);
                        bulk_commit_group();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_leader0 + 8u * acc);
        }
    }
    if (warp >= 2 && lane == 0) bulk_wait_group_all();
    __syncthreads();
    cluster_sync_all();  // no remote arrive or multicast is still pending
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512u);
    }
}

// ---------------------------------------------------------------- few rows
constexpr int kFewMaxStages = 12;
struct FewCtl {
    unsigned long long bar[2 * kFewMaxStages + 1];  // full, empty, done
    uint32_t tmem_base;
    int abort;
};

// One 128 (weight rows) x MT (rows of A) tile, K blocks [k0, k1) of it.
template <int MT>
__global__ void __launch_bounds__(NUM_THREADS)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const Fp8Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int X_BYTES = MT * BK;
    constexpr uint32_t TMEM_COLS = MT < 32 ? 32u : static_cast<uint32_t>(MT);
    const int S = p.stages;
    uint8_t* w_ring = smem;
    uint8_t* x_ring = smem + S * ROW_TILE_BYTES;
    FewCtl* ctl = reinterpret_cast<FewCtl*>(x_ring + S * X_BYTES);
    float* part = reinterpret_cast<float*>(smem);  // [MT][128], over the ring once it is read

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cl = static_cast<int>(blockIdx.x) / split;
    const int m0 = (cl % p.tiles_m) * MT, n0 = (cl / p.tiles_m) * 128;
    const int k0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / split);
    const int k1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / split);
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * S);
    volatile int* abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    griddep_launch_dependents();
    griddep_wait();

    int it = 0;  // thread 0: stages issued
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int kb = k0; kb < k1; ++kb, ++it) {
                if (!bounded_wait<false>(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns, ROLE_PRODUCER,
                                         it))
                    break;
                if (!(it == p.withhold && blockIdx.x == 0)) {
                    mbar_arrive_expect_tx(full_bar(s), ROW_TILE_BYTES + X_BYTES);
                    tma_load_2d(smem_addr(w_ring + s * ROW_TILE_BYTES), &tmW, full_bar(s), kb * BK, n0);
                    tma_load_2d(smem_addr(x_ring + s * X_BYTES), &tmX, full_bar(s), kb * BK, m0);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t w_desc0 = smem_desc(smem_addr(w_ring)), x_desc0 = smem_desc(smem_addr(x_ring));
        int s = 0;
        uint32_t ph = 0;
        for (int kb = k0; kb < k1; ++kb) {
            const bool r = bounded_wait<false>(full_bar(s), ph, abort_flag, p.wait_limit_ns, ROLE_MMA, kb - k0);
            if (!__all_sync(0xffffffffu, r)) break;
            tc_fence_after();
            const uint32_t w_off = static_cast<uint32_t>(s * ROW_TILE_BYTES) / 16u;
            const uint32_t x_off = static_cast<uint32_t>(s * X_BYTES) / 16u;
            if (elect_one_sync()) {
#pragma unroll
                for (int kk = 0; kk < BK / UMMA_K; ++kk)
                    umma_f8(tmem_base, w_desc0 + w_off + 2u * kk, x_desc0 + x_off + 2u * kk, p.idesc,
                            kb != k0 || kk != 0);
                umma_commit(empty_bar(s));
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
        // Also after an abort: every MMA this warp issued finishes here.
        if (elect_one_sync()) umma_commit(done_bar);
        __syncwarp();
        drain_wait(done_bar, 0u, p.wait_limit_ns);
        tc_fence_after();
        tc_fence_before();
    }
    __syncthreads();  // the accumulator is complete and the ring is read
    tc_fence_after();
    if (*abort_flag) {
        // Copies that no MMA waited for land before the ring is reused.
        if (threadIdx.x == 0)
            for (int j = it - S > 0 ? it - S : 0; j < it; ++j) {
                if (j == p.withhold && blockIdx.x == 0) continue;
                drain_wait(full_bar(j % S), static_cast<uint32_t>((j / S) & 1), p.wait_limit_ns);
            }
        __syncthreads();
    }
    if (warp >= 2) {
        const int q = warp & 3;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        const int n = 32 * q + lane;
#pragma unroll
        for (int c = 0; c < MT; c += 16) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_row + static_cast<uint32_t>(c), r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128 + n] = __uint_as_float(r[i]);
        }
        tc_fence_before();
    }
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // CTA `rank` adds the cluster's partials of its share of the rows, in rank
    // order, and writes them: a warp takes 128 outputs of one row.
    {
        const int rows = min(MT, p.M - m0);
        const int r0 = rows * rank / split, r1 = rows * (rank + 1) / split;
        const int n = n0 + 4 * lane;
        float bs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) bs[e] = n + e < p.N ? p.b_scale[n + e] : 0.0f;
        const uint32_t part_addr = smem_addr(part) + 16u * lane;
        for (int m = r0 + warp; m < r1; m += NUM_THREADS / 32) {
            const uint32_t at = part_addr + 512u * m;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (split == 1) {
                v = *reinterpret_cast<const float4*>(part + m * 128 + 4 * lane);
            } else {
                for (int c = 0; c < split; ++c) {
                    const float4 u = ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
            }
            const float as = p.a_scale[m0 + m];
            const uint32_t lo = pack16(v.x * as * bs[0], v.y * as * bs[1], p.out_bf16);
            const uint32_t hi = pack16(v.z * as * bs[2], v.w * as * bs[3], p.out_bf16);
            uint16_t* c = static_cast<uint16_t*>(p.C) + static_cast<long long>(m0 + m) * p.ldc + n;
            if (n + 4 <= p.N) {
                *reinterpret_cast<uint2*>(c) = make_uint2(lo, hi);
            } else {
                if (n < p.N) c[0] = static_cast<uint16_t>(lo);
                if (n + 1 < p.N) c[1] = static_cast<uint16_t>(lo >> 16);
                if (n + 2 < p.N) c[2] = static_cast<uint16_t>(hi);
            }
        }
    }
    if (split > 1) cluster_sync_all();  // the peers have read this CTA's partials
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Tensor map over a row-major matrix of `rows` x `cols` elements with row
// pitch ld_bytes: boxes of 128 bytes x box_rows, 128-byte swizzle, zero fill.
bool encode_rows(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t rows, uint64_t cols,
                 uint64_t ld_bytes, uint32_t box_cols, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld_bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_e4m3(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    return encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, cols, ld, BK, box_rows);
}

// Instruction descriptor (kind::f8f6f4): D fp32 (bit 4), A and B e4m3 (0 at
// bits 7 and 10), both K-major, N >> 3 at bits 17..22, M >> 4 at bits 24..28.
uint32_t instruction(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The kernels' dynamic shared-memory limit is set once a device.
bool allow_smem(const void* kernel, int slot) {
    static std::mutex mu;
    static bool done[64][8] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!done[dev][slot])
        done[dev][slot] =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) == cudaSuccess;
    return done[dev][slot];
}

struct Config {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Config(int64_t grid, int cluster, size_t smem, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(NUM_THREADS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
};

int resident_pairs() {
    static std::mutex mu;
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> g(mu);
    if (n[dev] == 0) {
        Config c(2, 2, kMaxSmem, nullptr);
        c.cfg.attrs = &c.attr[1];  // the cluster alone
        c.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n[dev], fp8_pair_kernel, &c.cfg) != cudaSuccess) n[dev] = 0;
    }
    return n[dev];
}

int finish(cudaError_t e) {
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

Fp8Params params_of(const Fp8Launch& L) {
    Fp8Params p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.K = static_cast<int>(L.K);
    p.k_blocks = static_cast<int>((L.K + BK - 1) / BK);
    p.out_bf16 = L.out_bf16;
    p.C = L.C;
    p.ldc = L.ldc;
    p.a_scale = L.a_scale;
    p.b_scale = L.b_scale;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    return p;
}

int launch_pair(const Fp8Launch& L, cudaStream_t stream) {
    Fp8Params p = params_of(L);
    p.tiles_m = static_cast<int>((L.M + 255) / 256);
    p.tiles_n = static_cast<int>((L.N + 255) / 256);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (tiles > (1 << 30)) return GEMM_ERR_UNSUPPORTED;
    // Tile rows walked together: about 32 MB of A, so that the panel stays in
    // L2 while the group walks its columns.
    const int64_t g = (32ll << 20) / (256 * L.K);
    p.group_m = static_cast<int>(g < 8 ? 8 : g > 16 ? 16 : g);
    p.stages = kPairStages;
    p.idesc = instruction(256, 256);
    CUtensorMap tmA, tmB, tmC;
    if (!encode_e4m3(&tmA, L.A, L.M, L.K, L.lda, 128) || !encode_e4m3(&tmB, L.B, L.N, L.K, L.ldb, 128) ||
        !encode_rows(&tmC, L.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, L.C,
                     L.M, L.N, L.ldc * 2, 64, 32))
        return GEMM_ERR_LAUNCH;
    if (!allow_smem(reinterpret_cast<const void*>(fp8_pair_kernel), 0)) return GEMM_ERR_LAUNCH;
    const int units = resident_pairs();
    if (units <= 0) return GEMM_ERR_LAUNCH;
    static_assert(1024 + 2 * kPairStages * ROW_TILE_BYTES + 4 * kPairBoxes * EPI_BOX_BYTES + sizeof(PairCtl) <=
                      kMaxSmem,
                  "the pair kernel's shared memory");
    Config c(2 * (tiles < units ? tiles : units), 2, kMaxSmem, stream);
    return finish(cudaLaunchKernelEx(&c.cfg, fp8_pair_kernel, tmA, tmB, tmC, p));
}

template <int MT>
int launch_few(const Fp8Launch& L, int slot, cudaStream_t stream) {
    Fp8Params p = params_of(L);
    constexpr int STAGE = ROW_TILE_BYTES + MT * BK;
    // Two CTAs an SM where a ring of four stages and the partials fit twice.
    constexpr bool kTwo = MT <= 64;
    constexpr int kBudget = (kTwo ? 112 : 226) * 1024;
    constexpr int kStages = (kBudget - 1024 - static_cast<int>(sizeof(FewCtl))) / STAGE;
    static_assert(kStages * STAGE >= MT * 128 * 4, "the partials lie over the ring");
    p.stages = kStages < kFewMaxStages ? kStages : kFewMaxStages;
    p.tiles_m = static_cast<int>((L.M + MT - 1) / MT);
    p.tiles_n = static_cast<int>((L.N + 127) / 128);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    const int sms = tc_current_device_sms();
    if (sms <= 0) return GEMM_ERR_CUDA;
    // Cut K over up to 8 CTAs while the grid stays within what is resident
    // at once and every CTA keeps four K blocks.
    int split = 1;
    while (split < 8 && tiles * split * 2 <= sms * (kTwo ? 2 : 1) && p.k_blocks / (2 * split) >= 4) split *= 2;
    p.split = split;
    if (tiles * split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    p.idesc = instruction(128, MT);
    CUtensorMap tmW, tmX;
    if (!encode_e4m3(&tmW, L.B, L.N, L.K, L.ldb, 128) || !encode_e4m3(&tmX, L.A, L.M, L.K, L.lda, MT))
        return GEMM_ERR_LAUNCH;
    auto kernel = fp8_few_kernel<MT>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), slot)) return GEMM_ERR_LAUNCH;
    Config c(tiles * split, split, 1024 + static_cast<size_t>(p.stages) * STAGE + sizeof(FewCtl), stream);
    return finish(cudaLaunchKernelEx(&c.cfg, kernel, tmW, tmX, p));
}

}  // namespace

int fp8_launch(const Fp8Launch& L, cudaStream_t stream) {
    if (L.M <= 16) return launch_few<16>(L, 1, stream);
    if (L.M <= 32) return launch_few<32>(L, 2, stream);
    if (L.M <= 64) return launch_few<64>(L, 3, stream);
    if (L.M <= 128) return launch_few<128>(L, 4, stream);
    if (L.M <= 256) return launch_few<256>(L, 5, stream);
    return launch_pair(L, stream);
}

int fp8_read_and_clear_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_fp8_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_fp8_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
