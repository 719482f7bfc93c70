// product_pair_sm103a.cu -- the products of a 16-bit linear layer for many rows:
// D = epilogue(A B) in 256 x 256 tiles on CTA pairs (tcgen05, cta_group::2).
//
// Persistent; two accumulators in tensor memory, so that a tile's epilogue runs
// under the next tile's mainloop.  Bound by the tensor pipe.  Either operand may
// be K-major or MN-major (product.cuh), so none is ever transposed in memory.
//
// The epilogue's inputs (a residual, a gradient, the z of an activation) come by
// tensor copies into the boxes that its outputs leave from: a box of 32 columns
// is filled up to four chunks ahead, changed in place and stored.
//
// Every wait is bounded (gemm_debug_set's limit, 2 s unless set): a wait that
// runs out records the failure, raises the pair's abort flags, lets the copies
// and products in flight land and ends.
#include <mutex>

#include "activation.cuh"
#include "product.cuh"

namespace ssp {

__device__ GemmDeviceStatus g_product_pair_status;

namespace {

constexpr int THREADS = 320;       // TMA warp, MMA warp, eight epilogue warps
constexpr int STAGES = 5;          // 32 KB each; a sixth would leave the epilogue one box a warp
constexpr int EPI_BYTES = 8192;    // boxes of an epilogue warp
constexpr uint16_t kPairMask = 0x3;

struct PairParams {
    int M, N;
    int tiles_m, tiles_n, tiles, k_blocks, batch;
    int k_chunks;  // accumulations of a tile, summed by the epilogue (EPI_F32)
    int group_m;   // tile rows walked together
    int a_mn, b_mn;
    uint32_t idesc;
    int act;
    int has_r, has_p;
    int symmetric;
    int clip;      // columns that tensor stores may write in units of 16 bytes
    float alpha, beta;
    const float* factor;
    int alpha_pow, beta_pow;
    const void* bias;
    // For boxes across the right edge, which each thread reads and writes itself.
    ProductMatrix D, R, P;
    unsigned long long wait_limit_ns;
    int withhold;
};

struct PairCtl {
    unsigned long long bar[2 * STAGES + 5];  // full, empty, tmem_full[2], tmem_empty[2], drain
    unsigned long long in_bar[8 * 4];        // inputs of an epilogue warp's boxes
    uint32_t tmem_base;
    int abort;
};
static_assert(1024 + 2 * STAGES * P_TILE_BYTES + 8 * EPI_BYTES + sizeof(PairCtl) <= kProductSmem, "shared memory");

// Output tile of persistent work item t: groups of group_m tile rows walked
// column by column, every other group backwards, so that the pairs running at
// one time share rows of A and columns of B in L2.  A symmetric result has its
// tiles on and below the diagonal alone, row by row.
__device__ __forceinline__ void tile_coords(const PairParams& p, int t, int& b, int& tm, int& tn) {
    b = t / p.tiles;
    t -= b * p.tiles;
    if (p.symmetric) {
        int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
        while ((i + 1) * (i + 2) / 2 <= t) ++i;
        while (i * (i + 1) / 2 > t) --i;
        tm = i;
        tn = t - i * (i + 1) / 2;
        return;
    }
    const int per_group = p.group_m * p.tiles_n;
    const int g = t / per_group;
    const int first_m = g * p.group_m;
    const int gsize = min(p.tiles_m - first_m, p.group_m);
    const int r = t - g * per_group;
    tm = first_m + r % gsize;
    tn = r / gsize;
    if (g & 1) tn = p.tiles_n - 1 - tn;
}

// Sixteen packed pairs of 16-bit values of this thread's row of a box.
__device__ __forceinline__ void read_box16(uint32_t buf, int lane, uint32_t (&u)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = ld_shared_v4(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
        u[4 * j] = v.x;
        u[4 * j + 1] = v.y;
        u[4 * j + 2] = v.z;
        u[4 * j + 3] = v.w;
    }
}
__device__ __forceinline__ void write_box16(uint32_t buf, int lane, const uint32_t (&u)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        st_shared_v4(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4),
                     make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]));
}

// The same of the first `left` columns of a row in global memory.
__device__ __forceinline__ void read_row16(const void* p, int left, uint32_t (&u)[16]) {
    const uint16_t* s = static_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t lo = 2 * i < left ? s[2 * i] : 0, hi = 2 * i + 1 < left ? s[2 * i + 1] : 0;
        u[i] = lo | (hi << 16);
    }
}
__device__ __forceinline__ void write_row16(void* p, int left, const uint32_t (&u)[16]) {
    uint16_t* d = static_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (2 * i < left) d[2 * i] = static_cast<uint16_t>(u[i]);
        if (2 * i + 1 < left) d[2 * i + 1] = static_cast<uint16_t>(u[i] >> 16);
    }
}

// A cluster of two CTAs computes a 256 x 256 tile.  CTA rank r stages rows
// 128r.. of the A tile and columns 128r.. of the B tile; both CTAs' copies of a
// stage complete on the leader's full[s]; the leader issues every MMA and its
// commits free the stage in both CTAs.  Each CTA's TMEM receives its own 128
// rows of the result.  BF16 is the type of the 16-bit tensors, of the output for
// EPI_STEP.
template <bool BF16, int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmR,
                        const __grid_constant__ CUtensorMap tmP, const PairParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* a_ring = smem;
    uint8_t* b_ring = smem + STAGES * P_TILE_BYTES;
    uint8_t* epi_ring = b_ring + STAGES * P_TILE_BYTES;
    PairCtl* ctl = reinterpret_cast<PairCtl*>(epi_ring + 8 * EPI_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1u;
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
    const int tiles = p.tiles * p.batch;
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    volatile int* abort_flag = &ctl->abort;
    // First K block of a tile's accumulation c.
    auto chunk_begin = [&](int c) { return EPI == EPI_F32 ? p.k_blocks * c / p.k_chunks : c * p.k_blocks; };
    const int chunks = EPI == EPI_F32 ? p.k_chunks : 1;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmD);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 16);  // one arrive per epilogue warp of both CTAs
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 32; ++i) mbar_init(smem_addr(&ctl->in_bar[i]), 1);
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
                int b, tm, tn;
                tile_coords(p, t, b, tm, tn);
                const int a_row = tm * 256 + static_cast<int>(rank) * 128;
                const int b_row = tn * 256 + static_cast<int>(rank) * 128;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!product_wait<true>(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns,
                                            &g_product_pair_status, P_PRODUCER, it)) {
                        ok = false;
                        break;
                    }
                    if (!(it == p.withhold && blockIdx.x == 0)) {
                        const uint32_t bar = leader_full0 + 8u * s;
                        if (leader) mbar_arrive_expect_tx(full_bar(s), 4u * P_TILE_BYTES);
                        const uint32_t a_dst = smem_addr(a_ring + s * P_TILE_BYTES);
                        const uint32_t b_dst = smem_addr(b_ring + s * P_TILE_BYTES);
                        if (p.a_mn) {
                            tma_load_3d_pair_hint(a_dst, &tmA, bar, a_row, kb * PK, b, a_policy);
                            tma_load_3d_pair_hint(a_dst + P_CHUNK_BYTES, &tmA, bar, a_row + 64, kb * PK, b, a_policy);
                        } else {
                            tma_load_3d_pair_hint(a_dst, &tmA, bar, kb * PK, a_row, b, a_policy);
                        }
                        if (p.b_mn) {
                            tma_load_3d_pair(b_dst, &tmB, bar, b_row, kb * PK, b);
                            tma_load_3d_pair(b_dst + P_CHUNK_BYTES, &tmB, bar, b_row + 64, kb * PK, b);
                        } else {
                            tma_load_3d_pair(b_dst, &tmB, bar, kb * PK, b_row, b);
                        }
                    }
                    ++it;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                if (leader) {
                    // Every copy this pair armed lands before the CTA exits.
                    for (int j = it - STAGES > 0 ? it - STAGES : 0; j < it; ++j) {
                        if (j == p.withhold && blockIdx.x == 0) continue;
                        drain_wait(full_bar(j % STAGES), static_cast<uint32_t>((j / STAGES) & 1), p.wait_limit_ns);
                    }
                } else {
                    // The peer's copies complete on the leader's barriers: a
                    // bounded grace period, then the closing cluster barrier
                    // keeps this CTA alive until the leader has drained.
                    const unsigned long long grace = p.wait_limit_ns < 200000ull ? p.wait_limit_ns : 200000ull;
                    const unsigned long long t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < grace) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint64_t a_desc0 = operand_desc(smem_addr(a_ring), p.a_mn);
            const uint64_t b_desc0 = operand_desc(smem_addr(b_ring), p.b_mn);
            const uint32_t a_step = operand_step(p.a_mn), b_step = operand_step(p.b_mn);
            int s = 0, it = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto mma_wait = [&](uint32_t bar, uint32_t parity) -> bool {
                const bool r = product_wait<true>(bar, parity, abort_flag, p.wait_limit_ns, &g_product_pair_status,
                                                  P_MMA, it);
                return __all_sync(0xffffffffu, r) != 0;
            };
            for (int t = unit; ok && t < tiles; t += units) {
                for (int c = 0; ok && c < chunks; ++c, ++lt) {
                    const int acc = lt & 1;
                    if (!mma_wait(tempty_bar(acc), static_cast<uint32_t>((lt >> 1) & 1) ^ 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
                    const int kb0 = chunk_begin(c), kb1 = chunk_begin(c + 1);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!mma_wait(full_bar(s), ph)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t off = static_cast<uint32_t>(s * P_TILE_BYTES) / 16u;
                        if (elect_one_sync()) {  // once a stage: an election costs about as much as a product
#pragma unroll
                            for (int kk = 0; kk < PK / PUMMA_K; ++kk)
                                umma_f16_pair(d_tmem, a_desc0 + (off + a_step * kk), b_desc0 + (off + b_step * kk),
                                              p.idesc, kb != kb0 || kk != 0);
                            umma_commit_pair_multicast(empty_bar(s), kPairMask);
                        }
                        __syncwarp();
                        ++it;
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (elect_one_sync()) umma_commit_pair_multicast(tfull_bar(acc), kPairMask);
                    __syncwarp();
                }
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
        const int half = (warp - 2) >> 2;  // two warps a quarter: columns 0..127 and 128..255 of the tile
        // Boxes of 32 rows by 32 columns.  A chunk takes one, or two where it has
        // a second input (z of the activation) or output (z kept, or the mirror
        // image of a symmetric result's); `depth` chunks have their own.
        constexpr int BOX = EPI == EPI_F32 ? 4096 : 2048;
        const int per_chunk = EPI == EPI_F32 ? 1
                              : EPI == EPI_LINEAR ? 1 + p.has_p
                              : EPI == EPI_GRAD   ? 1 + p.has_r
                                                  : 1 + p.symmetric;
        const int depth = EPI_BYTES / BOX / per_chunk;
        const uint32_t buf0 = smem_addr(epi_ring) + static_cast<uint32_t>((warp - 2) * EPI_BYTES);
        const uint32_t in_bar0 = smem_addr(&ctl->in_bar[(warp - 2) * 4]);
        const bool inputs = EPI == EPI_GRAD || p.has_r;
        const uint32_t in_bytes = static_cast<uint32_t>(BOX) * (EPI == EPI_GRAD && p.has_r ? 2u : 1u);
        const bool vec_bias = (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0;
        uint32_t in_phase = 0, in_pending = 0;  // bit d: parity of, and whether a copy is on its way to, chunk d's boxes
        uint32_t box = 0;  // chunks stored so far: their ring runs on from tile to tile
        int lt = 0;
        for (int t = unit; t < tiles; t += units) {
            int b, tm, tn;
            tile_coords(p, t, b, tm, tn);
            const int row_base = tm * 256 + static_cast<int>(rank) * 128 + 32 * q;
            const int col0 = tn * 256 + half * 128;
            const bool mirror = EPI == EPI_STEP && p.symmetric && tm != tn;
            int todo = 0;  // chunks of this warp within the result
            if (row_base < p.M && col0 < p.N) todo = min(4, (p.N - col0 + 31) / 32);
            // Tensor stores clip rows past M, and columns past N in units of 16
            // bytes: a box with part of such a unit is read and written by each
            // thread for its row.
            auto whole = [&](int ci) { return col0 + ci * 32 + 32 <= p.N || p.clip; };
            auto fetch = [&](int ci, uint32_t at) {  // lane 0: chunk ci's inputs
                const uint32_t bar = in_bar0 + 8u * at, buf = buf0 + at * per_chunk * BOX;
                mbar_arrive_expect_tx(bar, in_bytes);
                if (p.has_r) tma_load_3d(buf, &tmR, bar, col0 + ci * 32, row_base, b);
                if (EPI == EPI_GRAD) tma_load_3d(buf + (p.has_r ? BOX : 0), &tmP, bar, col0 + ci * 32, row_base, b);
            };
            if (inputs && todo > 0 && !*abort_flag) {
                if (lane == 0) bulk_wait_group_read<0>();  // the last tile's stores have read their boxes
                for (int ci = 0; ci < min(todo, depth); ++ci) {
                    if (!whole(ci)) continue;
                    const uint32_t at = (box + ci) % depth;
                    if (lane == 0) fetch(ci, at);
                    in_pending |= 1u << at;
                }
            }
            float alpha = 1.0f, beta = 1.0f;
            if constexpr (EPI == EPI_STEP) {
                alpha = p.alpha;
                beta = p.beta;
                if (p.factor) {
                    alpha *= power_of(p.factor, b, p.alpha_pow);
                    beta *= power_of(p.factor, b, p.beta_pow);
                }
            }
            if (EPI == EPI_LINEAR && p.bias && lane < 2) prefetch_l1(static_cast<const uint16_t*>(p.bias) + min(col0 + 64 * lane, p.N - 1));
            constexpr int KEPT = EPI == EPI_F32 ? 128 : 1;
            float kept[KEPT];
            bool ok = true;
            for (int c = 0; c < chunks; ++c, ++lt) {
                const int acc = lt & 1;
                const bool r = product_wait<true>(tfull_bar(acc), static_cast<uint32_t>((lt >> 1) & 1), abort_flag,
                                                  p.wait_limit_ns, &g_product_pair_status, P_EPILOGUE, lt);
                ok = __all_sync(0xffffffffu, r) != 0;
                if (!ok) break;
                tc_fence_after();
                if constexpr (EPI == EPI_F32) {
                    // This accumulation joins the others in registers, where a sum
                    // is rounded to nearest.
                    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                           static_cast<uint32_t>(acc * 256 + half * 128);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(t_row + 32u * i, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            kept[32 * i + e] = c ? kept[32 * i + e] + __uint_as_float(r[e]) : __uint_as_float(r[e]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty_leader0 + 8u * acc);
                }
            }
            if (!ok) break;
            const int acc = (lt - 1) & 1;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                   static_cast<uint32_t>(acc * 256 + half * 128);
            const int row = row_base + lane;
            auto chunk = [&](int ci, const float* sums) {
                const int n0 = col0 + ci * 32;
                const int left = p.N - n0;  // columns within the result, from n0
                const uint32_t at = box % depth;
                const uint32_t buf = buf0 + at * per_chunk * BOX;
                const bool tma = whole(ci);
                uint32_t r[32];
                if constexpr (EPI != EPI_F32) tmem_ld_32x32b_x32(t_row + 32u * ci, r);
                if (inputs && tma) {
                    if (product_wait<true>(in_bar0 + 8u * at, (in_phase >> at) & 1u, abort_flag, p.wait_limit_ns,
                                           &g_product_pair_status, P_EPILOGUE, lt)) {
                        in_phase ^= 1u << at;
                        in_pending &= ~(1u << at);
                    }
                }
                if (!inputs && lane == 0) {  // the store that last used these boxes has read them
                    if (depth == 4) bulk_wait_group_read<3>();
                    else bulk_wait_group_read<1>();
                }
                float v[32];
                if constexpr (EPI == EPI_F32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = sums[i];
                } else {
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
                __syncwarp();
                const bool mine = row < p.M;  // edge boxes: this thread's row is in the result
                auto element = [&](const ProductMatrix& m, int size) -> uint8_t* {
                    return const_cast<uint8_t*>(static_cast<const uint8_t*>(m.p)) +
                           (static_cast<long long>(b) * m.stride + static_cast<long long>(row) * m.ld + n0) * size;
                };
                if constexpr (EPI == EPI_F32) {
                    if (p.has_r) {
                        if (tma) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint4 u = ld_shared_v4(buf + lane * 128 + ((j ^ (lane & 7)) << 4));
                                v[4 * j] += __uint_as_float(u.x);
                                v[4 * j + 1] += __uint_as_float(u.y);
                                v[4 * j + 2] += __uint_as_float(u.z);
                                v[4 * j + 3] += __uint_as_float(u.w);
                            }
                        } else if (mine) {
                            const float* s = reinterpret_cast<const float*>(element(p.R, 4));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < left) v[i] += s[i];
                        }
                    }
                    if (tma) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared_v4(buf + lane * 128 + ((j ^ (lane & 7)) << 4),
                                         make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                    __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
                    } else if (mine) {
                        float* d = reinterpret_cast<float*>(element(p.D, 4));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < left) d[i] = v[i];
                    }
                } else {
                    if (EPI == EPI_LINEAR && p.bias) {
                        if (vec_bias && left >= 32) {
                            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + n0);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint4 u = s[j];
                                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = unpack16<BF16>(w[e]);
                                    v[8 * j + 2 * e] += f.x;
                                    v[8 * j + 2 * e + 1] += f.y;
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < left) v[i] += load16<BF16>(p.bias, n0 + i);
                        }
                    }
                    uint32_t u[16];
                    if (EPI == EPI_LINEAR && p.has_p) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = pack16<BF16>(v[2 * i], v[2 * i + 1]);
                        if (tma) write_box16(buf + BOX, lane, u);
                        else if (mine) write_row16(element(p.P, 2), left, u);
                    }
                    if constexpr (EPI == EPI_LINEAR)
                        with_activation(p.act, [&](auto a) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = activation<decltype(a)::value>(v[i]);
                        });
                    if constexpr (EPI == EPI_STEP) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= alpha;
                    }
                    if (p.has_r) {
                        if (tma) read_box16(buf, lane, u);
                        else if (mine) read_row16(element(p.R, 2), left, u);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 f = unpack16<(BF16 && EPI != EPI_STEP)>(u[i]);
                            if constexpr (EPI == EPI_STEP) {
                                v[2 * i] = fmaf(beta, f.x, v[2 * i]);
                                v[2 * i + 1] = fmaf(beta, f.y, v[2 * i + 1]);
                            } else {
                                v[2 * i] += f.x;
                                v[2 * i + 1] += f.y;
                            }
                        }
                    }
                    if constexpr (EPI == EPI_GRAD) {
                        if (tma) read_box16(buf + (p.has_r ? BOX : 0), lane, u);
                        else if (mine) read_row16(element(p.P, 2), left, u);
                        with_activation(p.act, [&](auto a) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 f = unpack16<BF16>(u[i]);
                                v[2 * i] *= derivative<decltype(a)::value>(f.x);
                                v[2 * i + 1] *= derivative<decltype(a)::value>(f.y);
                            }
                        });
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] = pack16<BF16>(v[2 * i], v[2 * i + 1]);
                    if (tma) write_box16(buf, lane, u);
                    else if (mine) write_row16(element(p.D, 2), left, u);
                    if (EPI == EPI_STEP && mirror) {
                        // Row e of the mirrored box is column n0 + e of this one.
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            st_shared_u16(buf + BOX + e * 64 + (((lane >> 3) ^ ((e >> 1) & 3)) << 4) + (lane & 7) * 2,
                                          static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1))));
                    }
                }
                if (!tma) return;
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmD, buf, n0, row_base, b);
                    if (EPI == EPI_LINEAR && p.has_p) tma_store_3d(&tmP, buf + BOX, n0, row_base, b);
                    if (EPI == EPI_STEP && mirror) tma_store_3d(&tmD, buf + BOX, row_base, n0, b);
                    bulk_commit_group();
                }
                // The box before this one is free once its store has read it: it
                // takes the inputs of the chunk that comes `depth` after its own.
                const int next = ci + depth - 1;
                if (inputs && ci >= 1 && next < todo && whole(next) && !*abort_flag) {
                    const uint32_t to = (box + depth - 1) % depth;
                    if (lane == 0) {
                        bulk_wait_group_read<1>();
                        fetch(next, to);
                    }
                    in_pending |= 1u << to;
                }
                ++box;
            };
            if constexpr (EPI == EPI_F32) {
#pragma unroll
                for (int ci = 0; ci < 4; ++ci)
                    if (ci < todo) chunk(ci, &kept[32 * ci]);
            } else {
#pragma unroll 1
                for (int ci = 0; ci < todo; ++ci) chunk(ci, nullptr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(tempty_leader0 + 8u * acc);
            }
        }
        // Inputs still on their way after an abort land before the CTA exits.
        if (lane == 0)
            for (int d = 0; d < depth; ++d)
                if ((in_pending >> d) & 1u) drain_wait(in_bar0 + 8u * d, (in_phase >> d) & 1u, p.wait_limit_ns);
    }
    if (warp >= 2 && lane == 0) bulk_wait_group_all();
    __syncthreads();
    cluster_sync_all();  // no remote arrive or multicast is still pending
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512u);
    }
}

// ---------------------------------------------------------------- host side
constexpr int kInstances = 7;

// The kernels' dynamic shared-memory limit is set once a device.
bool allow_smem(const void* kernel, int slot) {
    static std::mutex mu;
    static bool done[64][kInstances] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!done[dev][slot])
        done[dev][slot] =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem) == cudaSuccess;
    return done[dev][slot];
}

// CTA pairs that are resident at once (the instances alike).
int resident_pairs(const void* kernel) {
    static std::mutex mu;
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> g(mu);
    if (n[dev] == 0) {
        ProductConfig c(2, 2, THREADS, kProductSmem, nullptr);
        c.cfg.attrs = &c.attr[1];  // the cluster alone
        c.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n[dev], kernel, &c.cfg) != cudaSuccess) n[dev] = 0;
    }
    return n[dev];
}

template <bool BF16, int EPI>
int launch(const ProductLaunch& L, int slot, cudaStream_t stream) {
    PairParams p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.tiles_m = static_cast<int>((L.M + 255) / 256);
    p.tiles_n = static_cast<int>((L.N + 255) / 256);
    int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (L.symmetric) tiles = static_cast<int64_t>(p.tiles_m) * (p.tiles_m + 1) / 2;
    if (tiles * L.batch > (1 << 30)) return GEMM_ERR_UNSUPPORTED;
    p.tiles = static_cast<int>(tiles);
    p.batch = static_cast<int>(L.batch);
    p.k_blocks = static_cast<int>((L.K + PK - 1) / PK);
    p.k_chunks = EPI == EPI_F32 ? (p.k_blocks + kProductChunk - 1) / kProductChunk : 1;
    if (EPI == EPI_F32 && static_cast<int64_t>(p.k_blocks) * p.k_chunks > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    // Tile rows walked together: about 32 MB of A, so that the panel stays in
    // L2 while the group walks its columns.
    const int64_t g = (32ll << 20) / (512 * L.K);
    p.group_m = static_cast<int>(g < 8 ? 8 : g > 16 ? 16 : g);
    p.a_mn = L.a_mn;
    p.b_mn = L.b_mn;
    p.idesc = product_instruction(256, 256, L.bf16, L.a_mn, L.b_mn);
    p.act = L.act;
    p.has_r = L.R.p != nullptr;
    p.has_p = L.P.p != nullptr;
    p.symmetric = L.symmetric;
    constexpr int size = EPI == EPI_F32 ? 4 : 2;
    p.clip = L.padded || L.N % (16 / size) == 0;
    p.alpha = L.alpha;
    p.beta = L.beta;
    p.factor = L.factor;
    p.alpha_pow = L.alpha_pow;
    p.beta_pow = L.beta_pow;
    p.bias = L.bias;
    p.D = L.D;
    p.R = L.R;
    p.P = L.P;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    auto kernel = product_pair_kernel<BF16, EPI>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), slot)) return GEMM_ERR_LAUNCH;
    const int units = resident_pairs(reinterpret_cast<const void*>(kernel));
    if (units <= 0) return GEMM_ERR_LAUNCH;
    const int64_t all = tiles * L.batch;
    const int grid = static_cast<int>(2 * (all < units ? all : units));
    if (L.plan) {
        *L.plan = {LINEAR_KERNEL_PAIR, 256, 1, STAGES, grid, kProductSmem};
        return GEMM_OK;
    }
    const CUtensorMapDataType dt = EPI == EPI_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type16(BF16);
    const CUtensorMapDataType rt = EPI == EPI_STEP ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : dt;
    const CUtensorMapSwizzle sw = EPI == EPI_F32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const int64_t cols = L.padded ? (L.N + 7) / 8 * 8 : L.N;
    CUtensorMap tmA, tmB, tmD, tmR, tmP;
    if (!encode_operand(&tmA, L.A, L.a_mn, L.bf16, L.M, L.K, L.batch, 128) ||
        !encode_operand(&tmB, L.B, L.b_mn, L.bf16, L.N, L.K, L.batch, 128) ||
        !encode_matrices(&tmD, dt, size, sw, L.D, L.M, cols, L.batch, 32, 32))
        return GEMM_ERR_LAUNCH;
    tmR = tmP = tmD;
    if (L.R.p && !encode_matrices(&tmR, rt, size, sw, L.R, L.M, cols, L.batch, 32, 32)) return GEMM_ERR_LAUNCH;
    if (L.P.p && !encode_matrices(&tmP, dt, size, sw, L.P, L.M, cols, L.batch, 32, 32)) return GEMM_ERR_LAUNCH;
    ProductConfig c(grid, 2, THREADS, kProductSmem, stream);
    return product_finish(cudaLaunchKernelEx(&c.cfg, kernel, tmA, tmB, tmD, tmR, tmP, p));
}

}  // namespace

int product_pair_launch(const ProductLaunch& L, cudaStream_t stream) {
    switch (L.epi) {
        case EPI_LINEAR:
            return L.out_bf16 ? launch<true, EPI_LINEAR>(L, 0, stream) : launch<false, EPI_LINEAR>(L, 1, stream);
        case EPI_GRAD:
            return L.out_bf16 ? launch<true, EPI_GRAD>(L, 2, stream) : launch<false, EPI_GRAD>(L, 3, stream);
        case EPI_STEP:
            return L.out_bf16 ? launch<true, EPI_STEP>(L, 4, stream) : launch<false, EPI_STEP>(L, 5, stream);
        default: return launch<false, EPI_F32>(L, 6, stream);
    }
}

int product_pair_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_product_pair_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_product_pair_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
