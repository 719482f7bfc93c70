// product_pair_sm103a.cu -- the products of a 16-bit linear layer for many rows:
// D = epilogue(A B) in tiles of 256 rows by 192 to 256 columns on CTA pairs
// (tcgen05, cta_group::2).
//
// Persistent; two accumulators in tensor memory, so that a tile's epilogue runs
// under the next tile's mainloop.  Bound by the tensor pipe.  Either operand may
// be K-major or MN-major (product.cuh), so none is ever transposed in memory.
//
// Tiles are 192, 224 or 256 columns wide, as lets the pairs end together (choose, in
// product_few_sm103a.cu): 4096^3 is 256 tiles of 256 columns, four rounds of the 76
// pairs with the last a third full, or 304 tiles of 224, four full rounds of less work.
//
// An epilogue warp takes its 32 rows in boxes of 128-byte rows: 64 columns of 16
// bits, 32 of fp32.  Its inputs (a residual, a gradient, the z of an activation)
// come by tensor copies into the boxes that its outputs leave from.
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

constexpr int MAX_STAGES = 6;
constexpr int BOX = 4096;
constexpr int MOST_SLOTS = 4;      // boxes of an epilogue warp: two, or four
constexpr uint16_t kPairMask = 0x3;

// Warps: A's copies, MMA, B's copies, none, and eight of the epilogue.  Each
// operand has a warp for its copies, because issuing one keeps a thread for some
// 150 ns, and a stage's products take 240 to 270: 4096^3 takes 80 us so, and 86
// with one warp for both (dz^T x, two chunks an operand: 80 and 113).
constexpr int FIRST = 4;  // first warp of the epilogue
constexpr int THREADS = 32 * (FIRST + 8);

struct PairMaps {
    CUtensorMap A, A_edge, B, B_edge;
    CUtensorMap D, R, P;           // boxes of 128-byte rows
    CUtensorMap D32, R32, P32;     // of 32 columns: the last box of a tile of 224
    CUtensorMap mirror;            // the box a symmetric result's box is mirrored into
};

// t / d for t < 2^30 as t * by >> shift.  (A tile has a few such; the compiler's
// divisions took 0.3 us of the 1.9 that a plain tile's epilogue takes.)
struct Divisor {
    uint32_t by;
    int shift;
};
Divisor divisor(int64_t d) {
    int bits = 0;
    while ((int64_t{1} << bits) < d) ++bits;
    return {static_cast<uint32_t>(((int64_t{1} << (30 + bits)) + d - 1) / d), 30 + bits};
}
__device__ __forceinline__ int over(int t, Divisor d) {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(t)) * d.by) >> d.shift);
}

struct PairParams {
    int M, N;
    int bn;        // tile width
    int tiles_m, tiles_n, tiles, k_blocks, batch;
    int k_chunks;  // accumulations of a tile, summed by the epilogue (EPI_F32)
    int long_chunks;  // the first of them, of 2 kProductChunk blocks each; the others have kProductChunk
    int group_m;   // tile rows walked together
    Divisor by_tiles, by_group;            // tiles; those of a group
    Divisor by_rows, by_last_rows;         // a group's tile rows; the last group's
    int stages;
    int slots;     // boxes of an epilogue warp
    int a_mn, b_mn;
    int b_chunks;  // MN-major B: chunks of 64 columns of a CTA's stage
    int a_whole, b_whole;  // rows and columns below which a stage's chunks come by one copy
    uint32_t idesc;
    int act;
    int has_r, has_p;
    int symmetric;
    int n_copied;  // columns that leave by tensor stores, which clip in units of 16 bytes
    float alpha, beta;
    const float* factor;
    int alpha_pow, beta_pow;
    const void* bias;
    ProductMatrix D, P;  // for the last columns, which each thread writes itself
    unsigned long long wait_limit_ns;
    int withhold;
};

struct PairCtl {
    unsigned long long bar[2 * MAX_STAGES + 5];  // full, empty, tmem_full[2], tmem_empty[2], drain
    unsigned long long in_bar[8 * MOST_SLOTS];   // inputs of an epilogue warp's boxes
    uint32_t tmem_base;
    int abort;
};

// Output tile of persistent work item t: groups of group_m tile rows walked
// column by column, every other group backwards, so that the pairs running at
// one time share rows of A and columns of B in L2.  A symmetric result has its
// tiles on and below the diagonal alone, row by row.
__device__ __forceinline__ void tile_coords(const PairParams& p, int t, int& b, int& tm, int& tn) {
    b = over(t, p.by_tiles);
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
    const int g = over(t, p.by_group);
    const int first_m = g * p.group_m;
    const bool last = p.tiles_m - first_m < p.group_m;
    const int gsize = last ? p.tiles_m - first_m : p.group_m;
    const int r = t - g * per_group;
    tn = over(r, last ? p.by_last_rows : p.by_rows);
    tm = first_m + r - tn * gsize;
    if (g & 1) tn = p.tiles_n - 1 - tn;
}

// Where 16-byte piece j of this thread's row of a box lies: rows of 128 bytes, or
// (narrow) of 64.
__device__ __forceinline__ uint32_t piece_addr(uint32_t buf, int lane, int j, bool narrow = false) {
    return narrow ? buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4) : buf + lane * 128 + ((j ^ (lane & 7)) << 4);
}
// Thirty-two 16-bit values of it, in pairs, from the half h.
__device__ __forceinline__ void read_box(uint32_t buf, int lane, int h, bool narrow, uint32_t (&u)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = ld_shared_v4(piece_addr(buf, lane, 4 * h + j, narrow));
        u[4 * j] = v.x;
        u[4 * j + 1] = v.y;
        u[4 * j + 2] = v.z;
        u[4 * j + 3] = v.w;
    }
}
__device__ __forceinline__ void write_box(uint32_t buf, int lane, int h, bool narrow, const uint32_t (&u)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        st_shared_v4(piece_addr(buf, lane, 4 * h + j, narrow),
                     make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]));
}

// Those of thirty-two columns from n on that no tensor store writes: columns
// [n_copied, N) of this thread's row d, seven at most.
__device__ __forceinline__ void write_last(const PairParams& p, uint8_t* d, int n, const uint32_t (&u)[16]) {
    uint16_t* to = reinterpret_cast<uint16_t*>(d);
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (n + e >= p.n_copied && n + e < p.N) to[n + e] = static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1)));
}

// A cluster of two CTAs computes a 256 x bn tile.  CTA rank r stages rows 128r..
// of the A tile and columns (bn/2) r.. of the B tile; both CTAs' copies of a stage
// complete on the leader's full[s]; the leader issues every MMA and its commits
// free the stage in both CTAs.  Each CTA's TMEM receives its own 128 rows of the
// result.  BF16 is the type of the 16-bit tensors, of the output for EPI_STEP.
template <bool BF16, int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    product_pair_kernel(const __grid_constant__ PairMaps maps, const PairParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int S = p.stages;
    const int b_cols = p.bn / 2;  // columns of B that this CTA stages
    const int b_bytes = (p.b_mn ? 64 * p.b_chunks : b_cols) * PK * 2;
    uint8_t* a_ring = smem;
    uint8_t* b_ring = smem + S * P_TILE_BYTES;
    uint8_t* epi_ring = b_ring + S * b_bytes;
    PairCtl* ctl = reinterpret_cast<PairCtl*>(epi_ring + 8 * p.slots * BOX);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1u;
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
    const int tiles = p.tiles * p.batch;
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
    volatile int* abort_flag = &ctl->abort;
    const int chunks = EPI == EPI_F32 ? p.k_chunks : 1;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.A);
        tma_prefetch_desc(&maps.B);
        tma_prefetch_desc(&maps.D);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 16);  // one arrive per epilogue warp of both CTAs
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 8 * MOST_SLOTS; ++i) mbar_init(smem_addr(&ctl->in_bar[i]), 1);
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
    griddep_wait();
    griddep_launch_dependents();

    // 384 threads of 168 registers: 128 x 88 + 256 x 208 are as many.
    if (warp >= FIRST) {
        if constexpr (EPI == EPI_F32) registers_up<208>();
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t tempty_leader0 = mapa_shared(tempty_bar(0), 0u);
        // Two warps a quarter take turns at its boxes.  A box needs a second slot
        // beside its own for a second input (z of the activation) or output (z kept,
        // or the mirror image of a symmetric result's); `depth` boxes, a power
        // of two, have their own.
        const int half = (warp - FIRST) >> 2;
        constexpr int COLS = EPI == EPI_F32 ? 32 : 64;  // of a box
        const int boxes = (p.bn + COLS - 1) / COLS;     // of a tile; the last may have 32 columns
        const bool twin = EPI == EPI_LINEAR ? p.has_p : EPI == EPI_GRAD ? p.has_r : EPI == EPI_STEP ? p.symmetric : false;
        const int depth = twin ? p.slots / 2 : p.slots, size = twin ? 2 * BOX : BOX;
        const uint32_t buf0 = smem_addr(epi_ring) + static_cast<uint32_t>((warp - FIRST) * p.slots * BOX);
        const uint32_t in_bar0 = smem_addr(&ctl->in_bar[(warp - FIRST) * MOST_SLOTS]);
        const bool inputs = EPI == EPI_GRAD || p.has_r;
        const bool vec_bias = (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0;
        // Nothing but the sums: past all the branches below, which take as long as the
        // rounding.
        const bool plain = EPI == EPI_LINEAR && !p.bias && !p.has_p && !p.has_r && p.act == LINEAR_ACT_NONE;
        uint32_t in_phase = 0, in_pending = 0;  // bit d: parity of, and whether a copy is on its way to, slot d
        uint32_t count = 0;  // boxes stored so far: the slots run on from tile to tile
        int lt = 0;
        for (int t = unit; t < tiles; t += units) {
            int b, tm, tn;
            tile_coords(p, t, b, tm, tn);
            const int row_base = tm * 256 + static_cast<int>(rank) * 128 + 32 * q;
            const int row = row_base + lane;
            const int col0 = tn * p.bn;
            const bool mirror = EPI == EPI_STEP && p.symmetric && tm != tn;
            // Boxes half, half + 2, ... of the tile that lie within the result.
            const int within = row_base < p.M ? min(boxes, (p.N - col0 + COLS - 1) / COLS) : 0;
            auto width = [&](int box) { return min(COLS, p.bn - box * COLS); };
            auto fetch = [&](int box, uint32_t at) {  // lane 0: a box's inputs
                const uint32_t bar = in_bar0 + 8u * at, buf = buf0 + at * size;
                const int n = col0 + box * COLS;
                const bool narrow = EPI != EPI_F32 && width(box) == 32;
                const uint32_t bytes = narrow ? BOX / 2 : BOX;
                mbar_arrive_expect_tx(bar, EPI == EPI_GRAD && p.has_r ? 2u * bytes : bytes);
                if (p.has_r) tma_load_3d(buf, narrow ? &maps.R32 : &maps.R, bar, n, row_base, b);
                if (EPI == EPI_GRAD)
                    tma_load_3d(buf + (p.has_r ? BOX : 0), narrow ? &maps.P32 : &maps.P, bar, n, row_base, b);
            };
            if (inputs && half < within && !*abort_flag) {
                if (lane == 0) bulk_wait_group_read<0>();  // the last tile's stores have read their boxes
                for (int d = 0; d < depth; ++d) {
                    const int box = half + 2 * d;
                    if (box >= within) break;
                    const uint32_t at = (count + d) & (depth - 1);
                    if (lane == 0) fetch(box, at);
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
            if (EPI == EPI_LINEAR && p.bias && lane < 4)
                prefetch_l1(static_cast<const uint16_t*>(p.bias) + min(col0 + 64 * lane, p.N - 1));
            // This warp has read its part of the accumulator: its loads have returned
            // (tcgen05.wait::ld), so the arrival need not order other memory.  One that
            // does waits for the warp's stores, some 3000 clocks.
            auto release = [&](int acc) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader0 + 8u * acc);
            };
            constexpr int KEPT = EPI == EPI_F32 ? 4 : 1;
            float kept[KEPT][32];
            uint32_t t_row = 0;
            int acc = 0;
            bool ok = true;
            for (int c = 0; c < chunks; ++c, ++lt) {
                acc = lt & 1;
                const bool r = product_wait<true>(tfull_bar(acc), static_cast<uint32_t>((lt >> 1) & 1), abort_flag,
                                                  p.wait_limit_ns, &g_product_pair_status, P_EPILOGUE, lt);
                ok = __all_sync(0xffffffffu, r) != 0;
                if (!ok) break;
                tc_fence_after();
                t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * 256);
                if constexpr (EPI == EPI_F32) {
                    // An accumulation joins the others in registers, where a sum is
                    // rounded to nearest.
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (half + 2 * i < within) {
                            uint32_t r[32];
                            tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>((half + 2 * i) * 32), r);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                kept[i][e] = c ? kept[i][e] + __uint_as_float(r[e]) : __uint_as_float(r[e]);
                        }
                    }
                    release(acc);
                }
            }
            if (!ok) break;
            // Before a box's slot is written: its inputs are there, or the store
            // that last used it has read it.
            auto slot_ready = [&](uint32_t at) {
                if (inputs) {
                    if (product_wait<true>(in_bar0 + 8u * at, (in_phase >> at) & 1u, abort_flag, p.wait_limit_ns,
                                           &g_product_pair_status, P_EPILOGUE, lt)) {
                        in_phase ^= 1u << at;
                        in_pending &= ~(1u << at);
                    }
                }
                if (!inputs && lane == 0 && count >= static_cast<uint32_t>(depth)) {
                    if (depth == 2) bulk_wait_group_read<1>();  // (four slots are taken for inputs alone)
                    else bulk_wait_group_read<0>();
                }
                __syncwarp();
            };
            auto row_of = [&](const ProductMatrix& m, int size) -> uint8_t* {
                return const_cast<uint8_t*>(static_cast<const uint8_t*>(m.p)) +
                       (static_cast<long long>(b) * m.stride + static_cast<long long>(row) * m.ld) * size;
            };
            // After a box's store: the slot of this warp's box before it (or this one's
            // own, the only one) takes the inputs of the next that has none.
            auto stored = [&](int box) {
                const int next = depth == 1 ? box + 2 : box + 2 * (depth - 1);
                if (inputs && (depth == 1 || box >= 2) && next < within && !*abort_flag) {
                    const uint32_t to = (count + depth - 1) & (depth - 1);
                    if (lane == 0) {
                        if (depth == 1) bulk_wait_group_read<0>();
                        else bulk_wait_group_read<1>();
                        fetch(next, to);
                    }
                    in_pending |= 1u << to;
                }
                ++count;
            };
            if constexpr (EPI == EPI_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int box = half + 2 * i;
                    if (box < within) {
                        const int n0 = col0 + box * 32;
                        const uint32_t at = count & (depth - 1), buf = buf0 + at * size;
                        slot_ready(at);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t to = piece_addr(buf, lane, j);
                            if (p.has_r) {
                                const uint4 u = ld_shared_v4(to);
                                kept[i][4 * j] += __uint_as_float(u.x);
                                kept[i][4 * j + 1] += __uint_as_float(u.y);
                                kept[i][4 * j + 2] += __uint_as_float(u.z);
                                kept[i][4 * j + 3] += __uint_as_float(u.w);
                            }
                            st_shared_v4(to, make_uint4(__float_as_uint(kept[i][4 * j]), __float_as_uint(kept[i][4 * j + 1]),
                                                        __float_as_uint(kept[i][4 * j + 2]),
                                                        __float_as_uint(kept[i][4 * j + 3])));
                        }
                        if (n0 + 32 > p.n_copied && row < p.M) {
                            float* d = reinterpret_cast<float*>(row_of(p.D, 4));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (n0 + e >= p.n_copied && n0 + e < p.N) d[n0 + e] = kept[i][e];
                        }
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            if (n0 < p.n_copied) tma_store_3d(&maps.D, buf, n0, row_base, b);
                            bulk_commit_group();
                        }
                        stored(box);
                    }
                }
            } else {
                if (half >= within) release(acc);
#pragma unroll 1
                for (int box = half; box < within; box += 2) {
                    const int n0 = col0 + box * 64;
                    const bool narrow = width(box) == 32;
                    const uint32_t at = count & (depth - 1), buf = buf0 + at * size;
                    slot_ready(at);
                    // Thirty-two columns at a time, in a loop: unrolled, the four
                    // activations' code would be read from memory once a tile.
#pragma unroll 1
                    for (int h = 0; h < (narrow ? 1 : 2); ++h) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(box * 64 + 32 * h), r);
                        tmem_ld_wait();
                        if (box + 2 >= within && (narrow || h == 1)) release(acc);
                        const int n = n0 + 32 * h, left = p.N - n;  // columns within the result, from n
                        const bool last = n + 32 > p.n_copied && row < p.M && left > 0;
                        Pair v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = make_pair2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                        uint32_t u[16];
                        if (plain && !last) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = pack16<BF16>(v[e]);
                            write_box(buf, lane, h, narrow, u);
                            continue;
                        }
                        if (EPI == EPI_LINEAR && p.bias && left > 0) {
                            if (vec_bias && left >= 32) {
                                const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + n);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint4 x = s[j];
                                    u[4 * j] = x.x;
                                    u[4 * j + 1] = x.y;
                                    u[4 * j + 2] = x.z;
                                    u[4 * j + 3] = x.w;
                                }
                            } else {
                                const uint16_t* s = static_cast<const uint16_t*>(p.bias) + n;
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    u[e] = (2 * e < left ? s[2 * e] : 0u) |
                                           (2 * e + 1 < left ? static_cast<uint32_t>(s[2 * e + 1]) << 16 : 0u);
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = add2(v[e], unpack16_pair<BF16>(u[e]));
                        }
                        if (EPI == EPI_LINEAR && p.has_p) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = pack16<BF16>(v[e]);
                            write_box(buf + BOX, lane, h, narrow, u);
                            if (last) write_last(p, row_of(p.P, 2), n, u);
                        }
                        if constexpr (EPI == EPI_LINEAR)
                            with_activation(p.act, [&](auto a) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[e] = activation<decltype(a)::value>(v[e]);
                            });
                        if constexpr (EPI == EPI_STEP) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = mul2(v[e], pair_of(alpha));
                        }
                        if (p.has_r) {
                            read_box(buf, lane, h, narrow, u);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const Pair f = unpack16_pair<(BF16 && EPI != EPI_STEP)>(u[e]);
                                v[e] = EPI == EPI_STEP ? fma2(pair_of(beta), f, v[e]) : add2(v[e], f);
                            }
                        }
                        if constexpr (EPI == EPI_GRAD) {
                            read_box(buf + (p.has_r ? BOX : 0), lane, h, narrow, u);
                            with_activation(p.act, [&](auto a) {
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    v[e] = mul2(v[e], derivative<decltype(a)::value>(unpack16_pair<BF16>(u[e])));
                            });
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] = pack16<BF16>(v[e]);
                        write_box(buf, lane, h, narrow, u);
                        if (last) write_last(p, row_of(p.D, 2), n, u);
                        if (EPI == EPI_STEP && mirror) {
                            // Row e of the mirrored box is column n0 + e of this one.
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                st_shared_u16(buf + BOX + (32 * h + e) * 64 + (((lane >> 3) ^ ((e >> 1) & 3)) << 4) +
                                                  (lane & 7) * 2,
                                              static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1))));
                        }
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (n0 < p.n_copied) tma_store_3d(narrow ? &maps.D32 : &maps.D, buf, n0, row_base, b);
                        if (EPI == EPI_LINEAR && p.has_p && n0 < p.n_copied)
                            tma_store_3d(narrow ? &maps.P32 : &maps.P, buf + BOX, n0, row_base, b);
                        if (EPI == EPI_STEP && mirror) tma_store_3d(&maps.mirror, buf + BOX, row_base, n0, b);
                        bulk_commit_group();
                    }
                    stored(box);
                }
            }
        }
        // Inputs still on their way after an abort land before the CTA exits.
        if (lane == 0)
            for (int d = 0; d < depth; ++d)
                if ((in_pending >> d) & 1u) drain_wait(in_bar0 + 8u * d, (in_phase >> d) & 1u, p.wait_limit_ns);
    } else {
        if constexpr (EPI == EPI_F32) registers_down<88>();
        if (warp == 0 || warp == 2) {
            if (lane == 0) {
                const bool is_a = warp == 0;
                const uint32_t leader_full0 = mapa_shared(full_bar(0), 0u);
                const uint64_t a_policy = l2_policy_evict_last();  // A rows serve the whole group of columns
                const uint32_t ring = smem_addr(is_a ? a_ring : b_ring);
                const int bytes = is_a ? P_TILE_BYTES : b_bytes;
                const CUtensorMap* map = is_a ? &maps.A : &maps.B;
                int s = 0, it = 0;
                uint32_t ph = 0;
                bool ok = true;
                for (int t = unit; ok && t < tiles; t += units) {
                    int b, tm, tn;
                    tile_coords(p, t, b, tm, tn);
                    const int r0 = is_a ? tm * 256 + static_cast<int>(rank) * 128 : tn * p.bn + static_cast<int>(rank) * b_cols;
                    // The tile's stages, issue(shared address, barrier, k) for each.
                    auto stages = [&](auto issue) {
                        for (int kb = 0; kb < p.k_blocks; ++kb) {
                            if (!product_wait<true>(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns,
                                                    &g_product_pair_status, P_PRODUCER, it)) {
                                ok = false;
                                break;
                            }
                            if (!(it == p.withhold && blockIdx.x == 0)) {
                                // One arrive a stage: B's bytes may be counted before it.
                                if (leader && is_a) mbar_arrive_expect_tx(full_bar(s), 2u * (P_TILE_BYTES + b_bytes));
                                issue(ring + static_cast<uint32_t>(s * bytes), leader_full0 + 8u * s, kb * PK);
                            }
                            ++it;
                            if (++s == S) {
                                s = 0;
                                ph ^= 1u;
                            }
                        }
                    };
                    if (!(is_a ? p.a_mn : p.b_mn)) {
                        if (is_a)
                            stages([&](uint32_t dst, uint32_t bar, int k) {
                                tma_load_3d_pair_hint(dst, map, bar, k, r0, b, a_policy);
                            });
                        else
                            stages([&](uint32_t dst, uint32_t bar, int k) { tma_load_3d_pair(dst, map, bar, k, r0, b); });
                    } else if (r0 < (is_a ? p.a_whole : p.b_whole)) {  // the chunks lie within the matrix
                        stages([&](uint32_t dst, uint32_t bar, int k) { tma_load_4d_pair(dst, map, bar, r0, k, 0, b); });
                    } else {
                        const CUtensorMap* edge = is_a ? &maps.A_edge : &maps.B_edge;
                        const int n = is_a ? 2 : p.b_chunks;
                        stages([&](uint32_t dst, uint32_t bar, int k) {
                            for (int c = 0; c < n; ++c)
                                tma_load_3d_pair(dst + c * P_CHUNK_BYTES, edge, bar, r0 + 64 * c, k, b);
                        });
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
                    int kb = 0;
                    for (int c = 0; ok && c < chunks; ++c, ++lt) {
                        const int acc = lt & 1, kb0 = kb;
                        const int kb1 = EPI == EPI_F32 ? min(p.k_blocks, kb + (c < p.long_chunks ? 2 : 1) * kProductChunk)
                                                       : p.k_blocks;
                        if (!mma_wait(tempty_bar(acc), static_cast<uint32_t>((lt >> 1) & 1) ^ 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
                        for (; kb < kb1; ++kb) {
                            if (!mma_wait(full_bar(s), ph)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint32_t a_off = static_cast<uint32_t>(s * P_TILE_BYTES) / 16u;
                            const uint32_t b_off = static_cast<uint32_t>(s * b_bytes) / 16u;
                            if (elect_one_sync()) {  // once a stage: an election costs about as much as a product
    #pragma unroll
                                for (int kk = 0; kk < PK / PUMMA_K; ++kk)
                                    umma_f16_pair(d_tmem, a_desc0 + (a_off + a_step * kk), b_desc0 + (b_off + b_step * kk),
                                                  p.idesc, kb != kb0 || kk != 0);
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
                }
                if (!ok) {  // every MMA this warp issued finishes before TMEM is freed
                    if (elect_one_sync()) umma_commit_pair_multicast(drain_bar, 0x1);
                    __syncwarp();
                    if (lane == 0) drain_wait(drain_bar, 0u, p.wait_limit_ns);
                }
            }
            __syncwarp();
        }
    }
    if (warp >= FIRST && lane == 0) bulk_wait_group_read<0>();  // shared memory may go; the grid's end waits for the rest
    __syncthreads();
    cluster_sync_all();  // no remote arrive or multicast is still pending
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512u);
    }
}

// ---------------------------------------------------------------- host side
constexpr int kInstances = 7;

// K blocks of a tile whose epilogue outlasts its products.
constexpr int kShortSum = 10;

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
int launch(const ProductLaunch& L, int bn, int slot, cudaStream_t stream) {
    PairParams p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.bn = bn;
    p.tiles_m = static_cast<int>((L.M + 255) / 256);
    p.tiles_n = static_cast<int>((L.N + bn - 1) / bn);
    int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (L.symmetric) tiles = static_cast<int64_t>(p.tiles_m) * (p.tiles_m + 1) / 2;
    if (tiles * L.batch > (1 << 30)) return GEMM_ERR_UNSUPPORTED;
    p.tiles = static_cast<int>(tiles);
    p.batch = static_cast<int>(L.batch);
    p.k_blocks = static_cast<int>((L.K + PK - 1) / PK);
    // Accumulations of 512 rows; two of 1024 first where a sum is long enough for them to
    // cost it little precision (of 8192 rows 8e-7 of the norm for 6.5e-7), so that the
    // products run on under the last tile's epilogue (8192 x 4096 results of 8192 rows,
    // added in place: 302 us, with 512 all along 311).
    p.k_chunks = 1;
    if (EPI == EPI_F32) {
        p.long_chunks = p.k_blocks >= 12 * kProductChunk ? 2 : 0;
        p.k_chunks = p.long_chunks + (p.k_blocks - p.long_chunks * 2 * kProductChunk + kProductChunk - 1) / kProductChunk;
    }
    // Tile rows walked together: about 32 MB of A, so that the panel stays in
    // L2 while the group walks its columns.
    const int64_t g = (32ll << 20) / (512 * L.K);
    p.group_m = static_cast<int>(g < 8 ? 8 : g > 16 ? 16 : g);
    p.by_tiles = divisor(p.tiles);
    p.by_group = divisor(static_cast<int64_t>(p.group_m) * p.tiles_n);
    p.by_rows = divisor(p.group_m);
    p.by_last_rows = divisor(p.tiles_m % p.group_m ? p.tiles_m % p.group_m : p.group_m);
    p.a_mn = L.a_mn;
    p.b_mn = L.b_mn;
    p.b_chunks = (bn / 2 + 63) / 64;
    p.a_whole = p.M - 127;
    p.b_whole = p.N - (64 * p.b_chunks - 1);
    p.idesc = product_instruction(256, bn, L.bf16, L.a_mn, L.b_mn);
    // Four boxes an epilogue warp where a tile's products are over before an epilogue
    // that moves two tensors a box or adds to fp32, two elsewhere, and as many stages as
    // there is room for beside them.  (Sums of 512 added to 8192^2 fp32: 108 us, with two
    // boxes 122.  Where only outputs leave, three stages for five cost more than boxes
    // gain: the same without an addend 80 us, with two boxes 68.)
    const bool moves = (EPI == EPI_F32 || EPI == EPI_GRAD) && L.R.p;
    p.slots = moves && p.k_blocks <= kShortSum ? 4 : 2;
    const int stage = P_TILE_BYTES + (L.b_mn ? 64 * p.b_chunks : bn / 2) * PK * 2;
    const int room = kProductSmem - 1024 - 8 * p.slots * BOX - static_cast<int>(sizeof(PairCtl));
    static_assert((kProductSmem - 1024 - 16 * BOX - static_cast<int>(sizeof(PairCtl))) / (2 * P_TILE_BYTES) >= 5 &&
                      (kProductSmem - 1024 - 32 * BOX - static_cast<int>(sizeof(PairCtl))) / (2 * P_TILE_BYTES) >= 2,
                  "stages of the widest tile");
    p.stages = room / stage < MAX_STAGES ? room / stage : MAX_STAGES;
    p.act = L.act;
    p.has_r = L.R.p != nullptr;
    p.has_p = L.P.p != nullptr;
    p.symmetric = L.symmetric;
    constexpr int size = EPI == EPI_F32 ? 4 : 2;
    constexpr int unit = 16 / size;
    p.n_copied = L.padded ? (p.N + unit - 1) / unit * unit : p.N / unit * unit;
    p.alpha = L.alpha;
    p.beta = L.beta;
    p.factor = L.factor;
    p.alpha_pow = L.alpha_pow;
    p.beta_pow = L.beta_pow;
    p.bias = L.bias;
    p.D = L.D;
    p.P = L.P;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    auto kernel = product_pair_kernel<BF16, EPI>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), slot)) return GEMM_ERR_LAUNCH;
    const int units = product_resident_pairs();
    if (units <= 0) return GEMM_ERR_LAUNCH;
    const int64_t all = tiles * L.batch;
    const int grid = static_cast<int>(2 * (all < units ? all : units));
    if (L.plan) {
        *L.plan = {LINEAR_KERNEL_PAIR, 256, 1, p.stages, grid, kProductSmem};
        return GEMM_OK;
    }
    const CUtensorMapDataType dt = EPI == EPI_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type16(BF16);
    const CUtensorMapDataType rt = EPI == EPI_STEP ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : dt;
    PairMaps m = {};
    // Outputs end at the last whole 16 bytes of a row (a map of no columns, which
    // nothing uses, has one unit); inputs where the row ends.
    const int64_t out_cols = p.n_copied > 0 ? p.n_copied : unit;
    auto box = [&](CUtensorMap* map, const ProductMatrix& x, CUtensorMapDataType type, int64_t cols, int width, int rows) {
        return encode_matrices(map, type, size, width * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                               x, L.M, cols, L.batch, width, rows);
    };
    const int64_t p_cols = EPI == EPI_LINEAR ? out_cols : L.N;  // z kept, or read
    bool ok = encode_operand(&m.A, &m.A_edge, L.A, L.a_mn, L.bf16, L.M, L.K, L.batch, 128) &&
              encode_operand(&m.B, &m.B_edge, L.B, L.b_mn, L.bf16, L.N, L.K, L.batch, bn / 2) &&
              box(&m.D, L.D, dt, out_cols, 128 / size, 32);
    if (L.R.p) ok = ok && box(&m.R, L.R, rt, L.N, 128 / size, 32);
    if (L.P.p) ok = ok && box(&m.P, L.P, dt, p_cols, 128 / size, 32);
    if (size == 2 && bn % 64 != 0) {
        ok = ok && box(&m.D32, L.D, dt, out_cols, 32, 32);
        if (L.R.p) ok = ok && box(&m.R32, L.R, rt, L.N, 32, 32);
        if (L.P.p) ok = ok && box(&m.P32, L.P, dt, p_cols, 32, 32);
    }
    if (L.symmetric) ok = ok && box(&m.mirror, L.D, dt, out_cols, 32, 64);
    if (!ok) return GEMM_ERR_LAUNCH;
    ProductConfig c(grid, 2, THREADS, kProductSmem, stream);
    return product_finish(cudaLaunchKernelEx(&c.cfg, kernel, m, p));
}

}  // namespace

// CTA pairs that are resident at once (the instances alike).
int product_resident_pairs() {
    const void* kernel = reinterpret_cast<const void*>(product_pair_kernel<false, EPI_F32>);
    return allow_smem(kernel, 6) ? resident_pairs(kernel) : 0;
}

int product_pair_launch(const ProductLaunch& L, int bn, cudaStream_t stream) {
    switch (L.epi) {
        case EPI_LINEAR:
            return L.out_bf16 ? launch<true, EPI_LINEAR>(L, bn, 0, stream) : launch<false, EPI_LINEAR>(L, bn, 1, stream);
        case EPI_GRAD:
            return L.out_bf16 ? launch<true, EPI_GRAD>(L, bn, 2, stream) : launch<false, EPI_GRAD>(L, bn, 3, stream);
        case EPI_STEP:
            return L.out_bf16 ? launch<true, EPI_STEP>(L, bn, 4, stream) : launch<false, EPI_STEP>(L, bn, 5, stream);
        default: return launch<false, EPI_F32>(L, bn, 6, stream);
    }
}

int product_pair_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_product_pair_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_product_pair_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
