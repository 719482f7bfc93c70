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

#include <mutex>

#include "../../include/quant.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant.h"
#include "tensor_copy.cuh"

namespace ssp {

__device__ GemmDeviceStatus g_fp8_status;

namespace {

constexpr int BK = 128;                 // K of a stage: one 128-byte swizzle row of 8-bit values
constexpr int UMMA_K = 32;              // K per tcgen05.mma (kind::f8f6f4)
constexpr int ROW_TILE_BYTES = 128 * BK;  // 128 rows of a stage: 16 KB
constexpr int FEW_THREADS = 192;        // TMA warp, MMA warp, four epilogue warps
constexpr int PAIR_THREADS = 320;       // TMA warp, MMA warp, eight epilogue warps
constexpr int kMaxSmem = 227 * 1024;
constexpr int kPairMaxStages = 6;
constexpr int kPairBoxes = 2;           // output boxes per epilogue warp
constexpr int ROLE_PRODUCER = 0, ROLE_MMA = 1, ROLE_EPILOGUE = 2;

struct Fp8Params {
    int M, N, K;
    int tiles_m, tiles_n, k_blocks;
    int group_m;   // pair kernel: tile rows walked together
    int split;     // few-row kernel: CTAs of a cluster, each with a part of K
    int stages;
    uint32_t idesc;
    void* C;
    long long ldc;
    const float* a_scale;
    const float* b_scale;
    unsigned long long wait_limit_ns;
    int withhold;
};

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

// Two accumulators times a row's scale and their columns' scales, in 16 bits.
template <bool BF16>
__device__ __forceinline__ uint32_t scaled16(uint32_t a, uint32_t b, float2 row, float2 col) {
    uint64_t v, r, c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(row.x), "f"(row.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(col.x), "f"(col.y));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(r));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(c));
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
    if constexpr (BF16) {
        const __nv_bfloat162 o = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&o);
    } else {
        const __half2 o = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&o);
    }
}

// Four adjacent outputs of a row, of which `left` lie in it.
__device__ __forceinline__ void store_quad(uint16_t* c, int left, uint32_t lo, uint32_t hi) {
    if (left >= 4) {
        *reinterpret_cast<uint2*>(c) = make_uint2(lo, hi);
    } else {
        if (left > 0) c[0] = static_cast<uint16_t>(lo);
        if (left > 1) c[1] = static_cast<uint16_t>(lo >> 16);
        if (left > 2) c[2] = static_cast<uint16_t>(hi);
    }
}

// ---------------------------------------------------------------- many rows
struct PairCtl {
    unsigned long long bar[2 * kPairMaxStages + 5];  // full, empty, tmem_full[2], tmem_empty[2], drain
    uint32_t tmem_base;
    int abort;
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

// A cluster of two CTAs computes a 256 x 256 tile.  CTA rank r stages rows
// 128r.. of the A tile and weight rows 128r.. of the B tile; both CTAs' copies
// of a stage complete on the leader's full[s]; the leader issues every MMA and
// its commits free the stage in both CTAs.  Each CTA's TMEM receives its own
// 128 rows of C.
//
// S stages of 32 KB and output boxes of BOX_COLS columns share the 227 KB: six
// stages with boxes of 32 columns, or five with boxes of 64, whose tensor
// stores of whole 128-byte rows are fewer (see launch_pair).
template <bool BF16, int S, int BOX_COLS>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int EPI_BOX_BYTES = 32 * BOX_COLS * 2;
    uint8_t* a_ring = smem;
    uint8_t* b_ring = smem + S * ROW_TILE_BYTES;
    uint8_t* epi_ring = b_ring + S * ROW_TILE_BYTES;
    PairCtl* ctl = reinterpret_cast<PairCtl*>(epi_ring + 8 * kPairBoxes * EPI_BOX_BYTES);

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
            mbar_init(tempty_bar(a), 16);  // one arrive per epilogue warp of both CTAs
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
            const uint64_t a_desc0 = k_major_desc(smem_addr(a_ring));
            const uint64_t b_desc0 = k_major_desc(smem_addr(b_ring));
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
                    // One election a stage: electing a lane for every product
                    // costs about as many clocks (108) as the product (128).
                    if (elect_one_sync()) {
#pragma unroll
                        for (int kk = 0; kk < BK / UMMA_K; ++kk)
                            umma_f8_pair(d_tmem, a_desc0 + off + 2u * kk, b_desc0 + off + 2u * kk, p.idesc,
                                         (kb | kk) != 0);
                        umma_commit_pair_multicast(empty_bar(s), kPairMask);
                    }
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
        // Two warps a lane quarter: columns 0..127 and 128..255 of the tile.
        const int half = (warp - 2) >> 2;
        const uint32_t buf0 =
            smem_addr(epi_ring) + static_cast<uint32_t>((warp - 2) * kPairBoxes) * EPI_BOX_BYTES;
        const bool vec_scales = (reinterpret_cast<uintptr_t>(p.b_scale) & 15u) == 0;
        int lt = 0;
        uint32_t box = 0;  // boxes stored so far: their ring runs on from tile to tile
        for (int t = unit; t < tiles; t += units, ++lt) {
            const int acc = lt & 1;
            int tm, tn;
            tile_coords(p, t, tm, tn);
            const int row_base = tm * 256 + static_cast<int>(rank) * 128 + 32 * q;
            const int col0 = tn * 256;
            const float rs = row_base + lane < p.M ? p.a_scale[row_base + lane] : 0.0f;
            // The column scales are read as they are used, the same ones by every
            // lane: bring their lines closer meanwhile.
            if (lane < 4) prefetch_l1(p.b_scale + min(col0 + half * 128 + lane * 32, p.N - 1));
            const bool ok = bounded_wait<true>(tfull_bar(acc), static_cast<uint32_t>((lt >> 1) & 1), abort_flag,
                                               p.wait_limit_ns, ROLE_EPILOGUE, lt);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                   static_cast<uint32_t>(acc * 256 + half * 128);
            const float2 rs2 = make_float2(rs, rs);
            if (row_base < p.M) {
#pragma unroll 1
                for (int ci = 0; ci < 128 / BOX_COLS; ++ci) {
                    const int n0 = col0 + half * 128 + ci * BOX_COLS;  // the box's first column
                    if (n0 >= p.N) break;
                    const uint32_t buf = buf0 + (box % kPairBoxes) * EPI_BOX_BYTES;
                    uint32_t r[BOX_COLS];
#pragma unroll
                    for (int i = 0; i < BOX_COLS; i += 32)
                        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(ci * BOX_COLS + i),
                                           *reinterpret_cast<uint32_t(*)[32]>(&r[i]));
                    // The store that last used this box has read it.
                    if (lane == 0) bulk_wait_group_read<kPairBoxes - 1>();
                    float4 cs[BOX_COLS / 4];
                    if (vec_scales && n0 + BOX_COLS <= p.N) {
#pragma unroll
                        for (int i = 0; i < BOX_COLS / 4; ++i)
                            cs[i] = __ldg(reinterpret_cast<const float4*>(p.b_scale + n0) + i);
                    } else {
                        auto at = [&](int e) { return p.b_scale[min(n0 + e, p.N - 1)]; };
#pragma unroll
                        for (int i = 0; i < BOX_COLS / 4; ++i)
                            cs[i] = make_float4(at(4 * i), at(4 * i + 1), at(4 * i + 2), at(4 * i + 3));
                    }
                    tmem_ld_wait();
                    __syncwarp();
                    uint4 u[BOX_COLS / 8];
#pragma unroll
                    for (int jj = 0; jj < BOX_COLS / 8; ++jj) {
                        const float4 x = cs[2 * jj], y = cs[2 * jj + 1];
                        const uint32_t* v = &r[8 * jj];
                        u[jj] = make_uint4(scaled16<BF16>(v[0], v[1], rs2, make_float2(x.x, x.y)),
                                           scaled16<BF16>(v[2], v[3], rs2, make_float2(x.z, x.w)),
                                           scaled16<BF16>(v[4], v[5], rs2, make_float2(y.x, y.y)),
                                           scaled16<BF16>(v[6], v[7], rs2, make_float2(y.z, y.w)));
                    }
                    // Tensor stores clip rows past M, and columns past N in
                    // units of 16 bytes: a box with part of such a unit is
                    // written by each thread for its row.
                    if ((p.N & 7) == 0 || n0 + BOX_COLS <= p.N) {
                        // Chunk j of row r lies at j ^ (r & 7), in 64-byte rows at
                        // j ^ ((r >> 1) & 3).
                        const int turn = BOX_COLS == 64 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
                        for (int jj = 0; jj < BOX_COLS / 8; ++jj)
                            st_shared_v4(buf + lane * (BOX_COLS * 2) + ((jj ^ turn) << 4), u[jj]);
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tmC, buf, n0, row_base);
                            bulk_commit_group();
                        }
                        ++box;
                    } else if (row_base + lane < p.M) {
                        uint16_t* c = static_cast<uint16_t*>(p.C) +
                                      static_cast<long long>(row_base + lane) * p.ldc + n0;
#pragma unroll
                        for (int jj = 0; jj < BOX_COLS / 8; ++jj) {
                            const uint32_t w[4] = {u[jj].x, u[jj].y, u[jj].z, u[jj].w};
                            if (n0 + 8 * jj + 8 <= p.N) {
                                *reinterpret_cast<uint4*>(c + 8 * jj) = u[jj];
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (n0 + 8 * jj + e < p.N)
                                        c[8 * jj + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                            }
                        }
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
constexpr int kFewTwo = 64;   // widest MT of which two CTAs fit an SM
constexpr int kFewPush = 32;  // widest MT with room of its own for the cluster's partials
struct FewCtl {
    unsigned long long bar[2 * kFewMaxStages + 1];  // full, empty, done
    uint32_t tmem_base;
    int abort;
    alignas(16) float a_scale[256];
    alignas(16) float b_scale[128];
};
static_assert(sizeof(FewCtl) % 16 == 0, "pushed partials follow");

// One 128 (weight rows) x MT (rows of A) tile, K blocks [k0, k1) of it.
template <int MT, bool BF16>
__global__ void __launch_bounds__(FEW_THREADS)
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
    // Partials of a cut K.  PUSH: every CTA writes its share of each output to
    // the CTA that owns the output, in room of its own; a row's 32 quads (four
    // outputs) are dealt to the CTAs in runs.  Else they lie over the ring once
    // it is read and are fetched, with a second barrier until they have been.
    constexpr bool PUSH = MT <= kFewPush;
    float* part = reinterpret_cast<float*>(smem);  // [MT][128]
    const uint32_t recv = smem_addr(ctl + 1);

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
    if (PUSH && split > 1) cluster_arrive_relaxed();  // this CTA has started: its shared memory may be written to
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
        const uint64_t w_desc0 = k_major_desc(smem_addr(w_ring)), x_desc0 = k_major_desc(smem_addr(x_ring));
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
    } else {
        const int et = static_cast<int>(threadIdx.x) - 64;  // 0..127
        ctl->b_scale[et] = n0 + et < p.N ? p.b_scale[n0 + et] : 0.0f;
        for (int m = et; m < MT; m += 128) ctl->a_scale[m] = m0 + m < p.M ? p.a_scale[m0 + m] : 0.0f;
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
    const int rows = min(MT, p.M - m0);
    const int most = (32 + split - 1) / split;  // quads of an owner
    auto first = [&](int r) { return (32 * r + split - 1) / split; };
    if (PUSH && split > 1) cluster_wait();  // every CTA has started
    if (warp >= 2) {
        const int q = warp & 3;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        const int n = 32 * q + lane;
        const int quad = 8 * q + (lane & 7);  // split = 1: this thread's four columns
        const float4 bs = *reinterpret_cast<const float4*>(ctl->b_scale + 4 * quad);
        uint16_t* out = static_cast<uint16_t*>(p.C) + static_cast<long long>(m0) * p.ldc + n0 + 4 * quad;
        const int owner = (n >> 2) * split >> 5;
        const uint32_t push = PUSH && split > 1 ? mapa_shared(recv, static_cast<uint32_t>(owner)) +
                                                      16u * static_cast<uint32_t>(rank * rows * most + (n >> 2) - first(owner)) +
                                                      4u * (n & 3)
                                                : 0u;
#pragma unroll 2
        for (int c = 0; c < MT; c += 16) {
            if (c >= rows) break;
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_row + static_cast<uint32_t>(c), r);
            tmem_ld_wait();
            if (PUSH && split > 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < rows)
                        st_cluster_f32(push + 16u * static_cast<uint32_t>((c + i) * most), __uint_as_float(r[i]));
            } else if (split > 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * 128 + n] = __uint_as_float(r[i]);
            } else {
                // By way of shared memory, a warp its own, from a column a thread
                // to four adjacent outputs of four rows a thread.
                const uint32_t turn = smem_addr(part) + static_cast<uint32_t>(q * 4096 + (c & 16) * 128);
#pragma unroll
                for (int i = 0; i < 16; ++i) st_shared_u32(turn + static_cast<uint32_t>(i * 128 + lane * 4), r[i]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = c + 4 * i + (lane >> 3);
                    const uint4 v = ld_shared_v4(turn + static_cast<uint32_t>(i * 512 + lane * 16));
                    const float as = ctl->a_scale[m];
                    const float2 as2 = make_float2(as, as);
                    if (m < rows)
                        store_quad(out + static_cast<long long>(m) * p.ldc, p.N - n0 - 4 * quad,
                                   scaled16<BF16>(v.x, v.y, as2, make_float2(bs.x, bs.y)),
                                   scaled16<BF16>(v.z, v.w, as2, make_float2(bs.z, bs.w)));
                }
            }
        }
        tc_fence_before();
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync_all();
        // CTA `rank` adds the partials of its outputs in rank order, four
        // adjacent ones a thread.
        const int d0 = PUSH ? first(rank) : 0, count = PUSH ? first(rank + 1) - d0 : 32;
        const int i0 = PUSH ? 0 : rows * 32 * rank / split, i1 = PUSH ? rows * count : rows * 32 * (rank + 1) / split;
        const uint32_t part_addr = smem_addr(part);
        for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += FEW_THREADS) {
            const int m = i / count, d = d0 + i % count, n = n0 + 4 * d;
            float4 u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < split)
                    u[c] = ld_cluster_f4(PUSH ? mapa_shared(recv + 16u * static_cast<uint32_t>((c * rows + m) * most + d - d0),
                                                            static_cast<uint32_t>(rank))
                                              : mapa_shared(part_addr + 16u * i, static_cast<uint32_t>(c)));
            float4 v = u[0];
#pragma unroll
            for (int c = 1; c < 8; ++c)
                if (c < split) {
                    v.x += u[c].x;
                    v.y += u[c].y;
                    v.z += u[c].z;
                    v.w += u[c].w;
                }
            const float as = ctl->a_scale[m];
            const float4 bs = *reinterpret_cast<const float4*>(ctl->b_scale + 4 * d);
            const float2 as2 = make_float2(as, as);
            const uint32_t lo = scaled16<BF16>(__float_as_uint(v.x), __float_as_uint(v.y), as2, make_float2(bs.x, bs.y));
            const uint32_t hi = scaled16<BF16>(__float_as_uint(v.z), __float_as_uint(v.w), as2, make_float2(bs.z, bs.w));
            uint16_t* c = static_cast<uint16_t*>(p.C) + static_cast<long long>(m0 + m) * p.ldc + n;
            store_quad(c, p.N - n, lo, hi);
        }
    }
    if (!PUSH && split > 1) cluster_sync_all();  // the peers have read this CTA's partials
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- host side
bool encode_e4m3(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    return encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, base, rows, cols, ld, BK,
                       box_rows);
}

// Instruction descriptor (kind::f8f6f4): D fp32 (bit 4), A and B e4m3 (0 at
// bits 7 and 10), both K-major, N >> 3 at bits 17..22, M >> 4 at bits 24..28.
uint32_t instruction(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The kernels' dynamic shared-memory limit is set once a device.
bool allow_smem(const void* kernel, int slot) {
    static std::mutex mu;
    static bool done[64][16] = {};
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
    Config(int64_t grid, int cluster, int threads, size_t smem, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
};

// CTA pairs that are resident at once (the pair kernel's instances alike).
int resident_pairs(const void* kernel) {
    static std::mutex mu;
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> g(mu);
    if (n[dev] == 0) {
        Config c(2, 2, PAIR_THREADS, kMaxSmem, nullptr);
        c.cfg.attrs = &c.attr[1];  // the cluster alone
        c.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n[dev], kernel, &c.cfg) != cudaSuccess) n[dev] = 0;
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
    p.C = L.C;
    p.ldc = L.ldc;
    p.a_scale = L.a_scale;
    p.b_scale = L.b_scale;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    return p;
}

template <bool BF16, int S, int BOX_COLS>
int launch_pair_as(const Fp8Launch& L, int slot, cudaStream_t stream) {
    Fp8Params p = params_of(L);
    p.tiles_m = static_cast<int>((L.M + 255) / 256);
    p.tiles_n = static_cast<int>((L.N + 255) / 256);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (tiles > (1 << 30)) return GEMM_ERR_UNSUPPORTED;
    // Tile rows walked together: about 32 MB of A, so that the panel stays in
    // L2 while the group walks its columns.
    const int64_t g = (32ll << 20) / (256 * L.K);
    p.group_m = static_cast<int>(g < 8 ? 8 : g > 16 ? 16 : g);
    p.stages = S;
    p.idesc = instruction(256, 256);
    auto kernel = fp8_pair_kernel<BF16, S, BOX_COLS>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), slot)) return GEMM_ERR_LAUNCH;
    const int units = resident_pairs(reinterpret_cast<const void*>(kernel));
    if (units <= 0) return GEMM_ERR_LAUNCH;
    const int grid = static_cast<int>(2 * (tiles < units ? tiles : units));
    if (L.plan) {
        *L.plan = {QUANT_KERNEL_FP8_PAIR, 256, 1, S, grid, kMaxSmem};
        return GEMM_OK;
    }
    CUtensorMap tmA, tmB, tmC;
    if (!encode_e4m3(&tmA, L.A, L.M, L.K, L.lda, 128) || !encode_e4m3(&tmB, L.B, L.N, L.K, L.ldb, 128) ||
        !encode_rows(&tmC, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     BOX_COLS == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, L.C, L.M, L.N, L.ldc * 2,
                     BOX_COLS, 32))
        return GEMM_ERR_LAUNCH;
    static_assert(1024 + 2 * S * ROW_TILE_BYTES + 8 * kPairBoxes * 64 * BOX_COLS + sizeof(PairCtl) <= kMaxSmem,
                  "the pair kernel's shared memory");
    Config c(grid, 2, PAIR_THREADS, kMaxSmem, stream);
    return finish(cudaLaunchKernelEx(&c.cfg, kernel, tmA, tmB, tmC, p));
}

int launch_pair(const Fp8Launch& L, cudaStream_t stream) {
    // A short K ends in an epilogue sooner than a ring can run ahead: wider
    // boxes.  3000 x 5001 x 300: 17.7 us with five stages and 64 columns, 22.5
    // with six and 32; 2048^3 10.0 and 10.2; 4096^3 45.0 and 43.0;
    // 8191 x 28672 x 4096 509 and 496.
    if (L.K <= 2048)
        return L.out_bf16 ? launch_pair_as<true, 5, 64>(L, 0, stream) : launch_pair_as<false, 5, 64>(L, 1, stream);
    return L.out_bf16 ? launch_pair_as<true, 6, 32>(L, 12, stream) : launch_pair_as<false, 6, 32>(L, 13, stream);
}

template <int MT>
int launch_few(const Fp8Launch& L, int slot, int split, bool two, cudaStream_t stream) {
    Fp8Params p = params_of(L);
    constexpr int STAGE = ROW_TILE_BYTES + MT * BK;
    p.tiles_m = static_cast<int>((L.M + MT - 1) / MT);
    p.tiles_n = static_cast<int>((L.N + 127) / 128);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    p.split = split;
    if (tiles * split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    // Two CTAs an SM with half of shared memory each, or a ring as deep as one
    // CTA's room.
    const int budget = (two ? 112 : 226) * 1024;
    // Room for pushed partials: ceil(32/c) quads of a row from each of c CTAs.
    const int recv = MT <= kFewPush && split > 1 ? static_cast<int>(L.M < MT ? L.M : MT) * (32 + split) * 16 : 0;
    const int stages = (budget - 1024 - static_cast<int>(sizeof(FewCtl)) - recv) / STAGE;
    static_assert(4 * STAGE >= MT * 512, "other partials lie over the ring");
    p.stages = stages < kFewMaxStages ? stages : kFewMaxStages;
    p.idesc = instruction(128, MT);
    int smem = 1024 + p.stages * STAGE + static_cast<int>(sizeof(FewCtl)) + recv;
    if (smem < kTmemPairedSmem) smem = kTmemPairedSmem;
    static_assert(2 * kFewTwo <= 512 && MT <= 256, "two CTAs' tensor memory");
    if (L.plan) {
        *L.plan = {QUANT_KERNEL_FP8_FEW, MT, split, p.stages, static_cast<int>(tiles * split), smem};
        return GEMM_OK;
    }
    CUtensorMap tmW, tmX;
    if (!encode_e4m3(&tmW, L.B, L.N, L.K, L.ldb, 128) || !encode_e4m3(&tmX, L.A, L.M, L.K, L.lda, MT))
        return GEMM_ERR_LAUNCH;
    auto kernel = L.out_bf16 ? fp8_few_kernel<MT, true> : fp8_few_kernel<MT, false>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), 2 * slot + L.out_bf16)) return GEMM_ERR_LAUNCH;
    Config c(tiles * split, split, FEW_THREADS, smem, stream);
    return finish(cudaLaunchKernelEx(&c.cfg, kernel, tmW, tmX, p));
}

// Which kernel, tile and cut of K: the one with the least time by a model whose
// constants (microseconds) were fitted to every choice measured on 40 shapes of
// 1 to 5536 rows, 153 to 28672 columns and 82 to 8192 of K.  On 60 other shapes,
// drawn, its choices are 2 % slower than the best one of each on average, 22 %
// at most (541 x 1332 x 966: 7.0 us for 5.7).
//   * few rows: a round of resident CTAs takes each one's K blocks and an
//     epilogue that grows with MT, twice where two share an SM; a cut K adds the
//     partials' way through distributed shared memory, and rounds of clusters
//     after the first wait for whole clusters' room.  With half an SM a CTA
//     starts while the kernel before it ends, but its ring is half as deep:
//     4 x 2048 x 8192 takes 5.0 us so and 5.7 with a whole SM a CTA, 64 x 8192 x
//     8192 (K cut in two, one CTA an SM) 17.5 and 15.1.
//   * pairs: a round takes its K blocks at the tensor pipe's rate.
struct Choice {
    int mt = 0;  // 0: the pair kernel
    int split = 1;
    bool two = false;  // two CTAs an SM
};

// CTAs (one an SM) that the current device holds at once, by cluster size 1..8.
bool resident_ctas(int (&out)[9]) {
    static std::mutex mu;
    static bool known[64] = {};
    static int n[64][9] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const void* kernel = reinterpret_cast<const void*>(fp8_few_kernel<128, true>);
    if (!allow_smem(kernel, 9)) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!known[dev]) {
        for (int c = 1; c <= 8; ++c) {
            Config cfg(c, c, FEW_THREADS, 200 * 1024, nullptr);
            cfg.cfg.attrs = &cfg.attr[1];  // the cluster alone
            cfg.cfg.numAttrs = 1;
            int k = 0;
            if (cudaOccupancyMaxActiveClusters(&k, kernel, &cfg.cfg) != cudaSuccess) {
                cudaGetLastError();
                k = 0;
            }
            n[dev][c] = k * c;
        }
        if (n[dev][1] <= 0) return false;
        known[dev] = true;
    }
    for (int c = 0; c <= 8; ++c) out[c] = n[dev][c];
    return true;
}

bool choose(const Fp8Launch& L, Choice* best) {
    int resident[9];
    if (!resident_ctas(resident)) return false;
    const int64_t kb = (L.K + BK - 1) / BK;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t pairs = up(L.M, 256) * up(L.N, 256);
    double least = 3.4 + static_cast<double>(up(pairs, resident[2] > 1 ? resident[2] / 2 : 1)) * (0.3 * kb + 1.98);
    for (int mt = 16; mt <= 256 && (mt == 16 || mt < 2 * L.M); mt *= 2) {
        const int64_t tiles = up(L.M, mt) * up(L.N, 128);
        for (int c = 1; c <= 8 && c <= kb; ++c) {
            if (resident[c] <= 0) continue;
            const int64_t ctas = tiles * c;
            for (int t = 0; t <= (mt <= kFewTwo ? 1 : 0); ++t) {
                const double rounds = static_cast<double>(up(ctas, resident[c] * (1 + t)));
                const bool alone = ctas <= resident[c];  // one CTA an SM at most
                const double block = (t && alone ? 0.29 : 0.163) + 0.0009 * mt;
                const double us = (t ? 0.74 : 1.93) +
                                  rounds * (t && !alone ? 2.0 : 1.0) * (up(kb, c) * block + 0.69 + 0.012 * mt) +
                                  (c > 1 ? 1.17 + 0.0023 * mt + 0.08 * (rounds - 1.0) * c : 0.0);
                if (us < least) {
                    least = us;
                    *best = {mt, c, t == 1};
                }
            }
        }
    }
    return true;
}

}  // namespace

int fp8_launch(const Fp8Launch& L, cudaStream_t stream) {
    Choice c;
    if (!choose(L, &c)) return GEMM_ERR_CUDA;
    switch (c.mt) {
        case 16: return launch_few<16>(L, 1, c.split, c.two, stream);
        case 32: return launch_few<32>(L, 2, c.split, c.two, stream);
        case 64: return launch_few<64>(L, 3, c.split, c.two, stream);
        case 128: return launch_few<128>(L, 4, c.split, c.two, stream);
        case 256: return launch_few<256>(L, 5, c.split, c.two, stream);
        default: return launch_pair(L, stream);
    }
}

int fp8_read_and_clear_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_fp8_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_fp8_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
