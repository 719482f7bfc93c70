// product_few_sm103a.cu -- the products of a 16-bit linear layer for few rows, or
// few tiles: D = epilogue(A B) on single CTAs and clusters (tcgen05).
//
// The roles of the operands are exchanged: 128 columns of the result (rows of
// the weights) are the MMA's M side and MT = 16 to 256 rows its N side, so one
// row costs a 16-wide MMA instead of a 128-row tile that is empty but for one
// row.  K is cut over the CTAs of a cluster, whose fp32 partials meet in
// distributed shared memory and are added in rank order, so that a narrow product
// or a long sum still keeps every SM loading.  Bound by reading the operands.
//
// Sums of more than 512 rows a CTA for an fp32 result (product_few_kernel<MT, true>) are
// made in two accumulators in turn, which the epilogue's warps add up in registers under
// the products (kProductChunk), so they may be as long as they like.
//
// Every wait is bounded as in product_pair_sm103a.cu.
#include <mutex>

#include "activation.cuh"
#include "product.cuh"

namespace ssp {

__device__ GemmDeviceStatus g_product_few_status;

namespace {

constexpr int FIRST = 4;  // first epilogue warp, after the weights' copies, MMA, the rows' copies and none
// Warps.  Those that add up the accumulations keep 64 sums a thread at most.
template <int MT, bool SUMS>
constexpr int kWarps = FIRST + (SUMS ? (MT == 256 ? 16 : 8) : 4);
constexpr int kMaxStages = 12;
constexpr int kTwo = 64;   // widest MT of which two CTAs fit an SM
constexpr int kPush = 32;  // widest MT with room of its own for the cluster's partials

struct FewMaps {
    CUtensorMap F, F_edge, T, T_edge;
};

struct FewParams {
    int M, N;
    int tiles_m, tiles_n, k_blocks;
    int split;       // CTAs of a cluster, each with a part of K
    int stages;
    uint32_t tmem_cols;
    int f_mn, t_mn;  // the weights' side (columns of the result) and the rows'
    int f_whole, t_whole;  // columns and rows below which a stage's chunks come by one copy
    uint32_t idesc;
    int epi, act;
    int bf16;        // type of the 16-bit tensors, of the output for EPI_STEP
    float alpha, beta;
    const float* factor;
    int alpha_pow, beta_pow;
    const void* bias;
    ProductMatrix D, R, P;
    unsigned long long wait_limit_ns;
    int withhold;
};

struct FewCtl {
    unsigned long long bar[2 * kMaxStages + 5];  // full, empty, done; accumulators full and empty
    uint32_t tmem_base;
    int abort;
    alignas(16) float bias[128];  // of the tile's columns
};
static_assert(sizeof(FewCtl) % 16 == 0, "pushed partials follow");

__device__ __forceinline__ long long place(const ProductMatrix& m, int b, int row, int n) {
    return static_cast<long long>(b) * m.stride + static_cast<long long>(row) * m.ld + n;
}

// Eight adjacent 16-bit elements of a row, of which `left` lie in it.
__device__ __forceinline__ uint4 load_eight(const void* p, long long i, int left) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
    if (left >= 8) return *reinterpret_cast<const uint4*>(s);
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = 2 * k < left ? s[2 * k] : 0, hi = 2 * k + 1 < left ? s[2 * k + 1] : 0;
        u[k] = lo | (hi << 16);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void store_eight(bool bf16, const void* p, long long i, int left, const Pair (&v)[4]) {
    uint16_t* d = static_cast<uint16_t*>(const_cast<void*>(p)) + i;
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = both(v[k]);
        u[k] = pack16(bf16, f.x, f.y);
    }
    if (left >= 8) {
        *reinterpret_cast<uint4*>(d) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (k < left) d[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1)));
    }
}

__device__ __forceinline__ void unpack_eight(bool bf16, uint4 u, Pair (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 x = unpack16(bf16, w[k]);
        f[k] = make_pair2(x.x, x.y);
    }
}

// The epilogue of eight adjacent sums v of row `row` from column n on; `bias` is the
// shared-memory address of the columns'.  Both its callers call it in a loop that
// is not unrolled: its code is long, runs once a CTA, and eight copies of it took
// 8 us to be read and run for 64 rows, one takes 2.
template <bool SUMS>
__device__ __forceinline__ void finish_eight(const FewParams& p, int b, int row, int n, Pair (&v)[4], uint32_t bias,
                                             float alpha, float beta) {
    const int left = p.N - n;
    if (left <= 0) return;
    if (SUMS || p.epi == EPI_F32) {
        float* d = static_cast<float*>(const_cast<void*>(p.D.p)) + place(p.D, b, row, n);
        const float* r = p.R.p ? static_cast<const float*>(p.R.p) + place(p.R, b, row, n) : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 x = both(v[2 * h]), y = both(v[2 * h + 1]);
            float4 o = make_float4(x.x, x.y, y.x, y.y);
            if (left >= 4 * h + 4) {
                if (r) {
                    const float4 u = *reinterpret_cast<const float4*>(r + 4 * h);
                    o = make_float4(o.x + u.x, o.y + u.y, o.z + u.z, o.w + u.w);
                }
                *reinterpret_cast<float4*>(d + 4 * h) = o;
            } else {
                if (left > 4 * h) d[4 * h] = r ? o.x + r[4 * h] : o.x;
                if (left > 4 * h + 1) d[4 * h + 1] = r ? o.y + r[4 * h + 1] : o.y;
                if (left > 4 * h + 2) d[4 * h + 2] = r ? o.z + r[4 * h + 2] : o.z;
            }
        }
        return;
    }
    const bool bf16 = p.bf16 != 0;
    // What is read beside the sums, asked for together.
    uint4 ru = {}, pu = {};
    if (p.R.p) ru = load_eight(p.R.p, place(p.R, b, row, n), left);
    if (p.epi == EPI_GRAD) pu = load_eight(p.P.p, place(p.P, b, row, n), left);
    Pair f[4];
    if (p.epi == EPI_LINEAR) {
        const uint4 lo = ld_shared_v4(bias), hi = ld_shared_v4(bias + 16);
        v[0] = add2(v[0], make_pair2(__uint_as_float(lo.x), __uint_as_float(lo.y)));
        v[1] = add2(v[1], make_pair2(__uint_as_float(lo.z), __uint_as_float(lo.w)));
        v[2] = add2(v[2], make_pair2(__uint_as_float(hi.x), __uint_as_float(hi.y)));
        v[3] = add2(v[3], make_pair2(__uint_as_float(hi.z), __uint_as_float(hi.w)));
        if (p.P.p) store_eight(bf16, p.P.p, place(p.P, b, row, n), left, v);
        with_activation(p.act, [&](auto a) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = activation<decltype(a)::value>(v[k]);
        });
    }
    if (p.epi == EPI_STEP) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], pair_of(alpha));
    }
    if (p.R.p) {
        unpack_eight(bf16 && p.epi != EPI_STEP, ru, f);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fma2(pair_of(beta), f[k], v[k]);
    }
    if (p.epi == EPI_GRAD) {
        unpack_eight(bf16, pu, f);
        with_activation(p.act, [&](auto a) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], derivative<decltype(a)::value>(f[k]));
        });
    }
    store_eight(bf16, p.D.p, place(p.D, b, row, n), left, v);
}

// One 128 (columns) x MT (rows) tile, a part of its K blocks.  SUMS: fp32 results, two
// accumulators of kProductChunk blocks at most in turn.
template <int MT, bool SUMS>
__global__ void __launch_bounds__(32 * kWarps<MT, SUMS>, MT <= kTwo ? 2 : 1)
    product_few_kernel(const __grid_constant__ FewMaps maps, const FewParams p) {
    constexpr int WARPS = kWarps<MT, SUMS>, THREADS = 32 * WARPS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int T_BYTES = MT * PK * 2;
    const int S = p.stages;
    uint8_t* f_ring = smem;
    uint8_t* t_ring = smem + S * P_TILE_BYTES;
    FewCtl* ctl = reinterpret_cast<FewCtl*>(t_ring + S * T_BYTES);
    // Partials of a cut K.  PUSH: every CTA writes its share of each output to
    // the CTA that owns the output, in room of its own; a row's 16 groups of eight
    // outputs are dealt to the CTAs in runs.  Else they lie over the ring once
    // it is read and are fetched, with a second barrier until they have been.
    constexpr bool PUSH = MT <= kPush;
    // When the next launch's CTAs may start: once the products are done, so that they
    // spread over the SMs as these leave, or, where a call is little but its start,
    // as soon as the launch before has ended (in graphs, 1 x 4096 x 4096: 8.05 us so, 8.2
    // late; six 2048 x 512 orthogonalised: 165 us late, 169 so).
    constexpr bool LATE = MT > 16;
    float* part = reinterpret_cast<float*>(smem);  // [MT][128]
    const uint32_t recv = smem_addr(ctl + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    int cl = static_cast<int>(blockIdx.x) / split;
    const int b = cl / (p.tiles_m * p.tiles_n);
    cl -= b * (p.tiles_m * p.tiles_n);
    const int m0 = (cl % p.tiles_m) * MT, n0 = (cl / p.tiles_m) * 128;
    const int k0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / split);
    const int k1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / split);
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * S);
    auto acc_full = [&](int a) { return bar0 + 8u * (2 * S + 1 + a); };
    auto acc_empty = [&](int a) { return bar0 + 8u * (2 * S + 3 + a); };
    volatile int* abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        if (p.k_blocks) {
            tma_prefetch_desc(&maps.F);
            tma_prefetch_desc(&maps.T);
        }
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        for (int a = 0; SUMS && a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_empty(a), WARPS - FIRST);
        }
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&ctl->tmem_base), p.tmem_cols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    if (PUSH && split > 1) cluster_arrive_relaxed();  // this CTA has started: its shared memory may be written to
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    griddep_wait();
    if (!LATE) griddep_launch_dependents();

    // SUMS: a warp of the epilogue has a quarter of the columns, a thread each, and ROWS of
    // the rows.
    constexpr int ROWS = SUMS ? MT / ((WARPS - FIRST) / 4) : 16;
    const int row0 = SUMS ? (warp - FIRST) / 4 * ROWS : 0;
    float kept[ROWS] = {};

    int it = 0;  // the copying threads: stages issued
    if (warp == 0 || warp == 2) {
        if (lane == 0) {
            const bool weights = warp == 0;
            const uint32_t ring = smem_addr(weights ? f_ring : t_ring);
            const uint32_t bytes = weights ? P_TILE_BYTES : T_BYTES;
            const CUtensorMap* map = weights ? &maps.F : &maps.T;
            const int r0 = weights ? n0 : m0;
            auto stages = [&](auto issue) {
                int s = 0;
                uint32_t ph = 0;
                for (int kb = k0; kb < k1; ++kb, ++it) {
                    if (!product_wait<false>(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns, &g_product_few_status,
                                             P_PRODUCER, it))
                        break;
                    if (!(it == p.withhold && blockIdx.x == 0)) {
                        // One arrive a stage: the rows' bytes may be counted before it.
                        if (weights) mbar_arrive_expect_tx(full_bar(s), P_TILE_BYTES + T_BYTES);
                        issue(ring + static_cast<uint32_t>(s) * bytes, full_bar(s), kb * PK);
                    }
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            };
            if (!(weights ? p.f_mn : p.t_mn)) {
                stages([&](uint32_t dst, uint32_t bar, int k) { tma_load_3d(dst, map, bar, k, r0, b); });
            } else if (r0 < (weights ? p.f_whole : p.t_whole)) {  // the chunks lie within the matrix
                stages([&](uint32_t dst, uint32_t bar, int k) { tma_load_4d(dst, map, bar, r0, k, 0, b); });
            } else {
                const CUtensorMap* edge = weights ? &maps.F_edge : &maps.T_edge;
                const int n = weights ? 2 : MT / 64;
                stages([&](uint32_t dst, uint32_t bar, int k) {
                    for (int c = 0; c < n; ++c) tma_load_3d(dst + c * P_CHUNK_BYTES, edge, bar, r0 + 64 * c, k, b);
                });
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t f_desc0 = operand_desc(smem_addr(f_ring), p.f_mn);
        const uint64_t t_desc0 = operand_desc(smem_addr(t_ring), p.t_mn);
        const uint32_t f_step = operand_step(p.f_mn), t_step = operand_step(p.t_mn);
        int s = 0;
        uint32_t ph = 0;
        auto mma_wait = [&](uint32_t bar, uint32_t parity, int kb) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
            const bool r = product_wait<false>(bar, parity, abort_flag, p.wait_limit_ns, &g_product_few_status, P_MMA,
                                               kb - k0);
            return __all_sync(0xffffffffu, r) != 0;
        };
        bool ok = true;
        for (int kb = k0, c = 0; ok && kb < k1; ++c) {  // accumulations
            const int kb0 = kb, kb1 = SUMS ? min(k1, kb + kProductChunk) : k1;
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(SUMS ? (c & 1) * MT : 0);
            if constexpr (SUMS) {
                ok = mma_wait(acc_empty(c & 1), static_cast<uint32_t>((c >> 1) & 1) ^ 1u, kb);
                if (!ok) break;
                tc_fence_after();
            }
            for (; kb < kb1; ++kb) {
                ok = mma_wait(full_bar(s), ph, kb);
                if (!ok) break;
                tc_fence_after();
                const uint32_t f_off = static_cast<uint32_t>(s * P_TILE_BYTES) / 16u;
                const uint32_t t_off = static_cast<uint32_t>(s * T_BYTES) / 16u;
                if (elect_one_sync()) {
#pragma unroll
                    for (int kk = 0; kk < PK / PUMMA_K; ++kk)
                        umma_f16(d_tmem, f_desc0 + (f_off + f_step * kk), t_desc0 + (t_off + t_step * kk), p.idesc,
                                 kb != kb0 || kk != 0);
                    umma_commit(empty_bar(s));
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if constexpr (SUMS) {
                if (ok && elect_one_sync()) umma_commit(acc_full(c & 1));
                __syncwarp();
            }
        }
        // Also after an abort: every MMA this warp issued finishes here.
        if (elect_one_sync()) umma_commit(done_bar);
        __syncwarp();
        drain_wait(done_bar, 0u, p.wait_limit_ns);
        tc_fence_after();
        tc_fence_before();
    } else if (warp >= FIRST) {
        const int et = static_cast<int>(threadIdx.x) - 32 * FIRST;  // 0..127, more for SUMS
        if (!SUMS) ctl->bias[et] = p.bias && n0 + et < p.N ? load16(p.bf16 != 0, p.bias, n0 + et) : 0.0f;
        // What this CTA's epilogue will read comes closer meanwhile, a line a thread.
        if (p.R.p || p.epi == EPI_GRAD) {
            const int rows = min(MT, p.M - m0);
            const int own0 = PUSH ? 0 : rows * rank / split, own1 = PUSH ? rows : rows * (rank + 1) / split;
            const int size = p.epi == EPI_F32 ? 4 : 2, lines = size;  // 128 columns a row
            for (int i = et; i < (own1 - own0) * lines; i += THREADS - 32 * FIRST) {
                const int m = m0 + own0 + i / lines, n = min(n0 + i % lines * (128 / size), p.N - 1);
                if (p.R.p) prefetch_l1(static_cast<const uint8_t*>(p.R.p) + place(p.R, b, m, n) * size);
                if (p.epi == EPI_GRAD) prefetch_l1(static_cast<const uint8_t*>(p.P.p) + place(p.P, b, m, n) * size);
            }
        }
        if constexpr (SUMS) {
            const uint32_t mine = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + static_cast<uint32_t>(row0);
            const int chunks = (k1 - k0 + kProductChunk - 1) / kProductChunk;
            for (int c = 0; c < chunks; ++c) {
                const bool w = product_wait<false>(acc_full(c & 1), static_cast<uint32_t>((c >> 1) & 1), abort_flag,
                                                   p.wait_limit_ns, &g_product_few_status, P_EPILOGUE, c);
                if (!__all_sync(0xffffffffu, w)) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < ROWS; i += 16) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(mine + static_cast<uint32_t>((c & 1) * MT + i), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) kept[i + e] += __uint_as_float(r[e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty(c & 1));
            }
        }
    }
    __syncthreads();  // the accumulators are complete and the ring is read
    if (LATE) griddep_launch_dependents();
    tc_fence_after();
    if (*abort_flag) {
        // Copies that no MMA waited for land before the ring is reused.  (A stage
        // that only one of the two warps issued is waited for until the limit.)
        if (lane == 0 && (warp == 0 || warp == 2))
            for (int j = it - S > 0 ? it - S : 0; j < it; ++j) {
                if (j == p.withhold && blockIdx.x == 0) continue;
                drain_wait(full_bar(j % S), static_cast<uint32_t>((j / S) & 1), p.wait_limit_ns);
            }
        __syncthreads();
    }
    float alpha = 1.0f, beta = 1.0f;
    if (p.epi == EPI_STEP) {
        alpha = p.alpha;
        beta = p.beta;
        if (p.factor) {
            alpha *= power_of(p.factor, b, p.alpha_pow);
            beta *= power_of(p.factor, b, p.beta_pow);
        }
    }
    const int rows = min(MT, p.M - m0);
    const int most = (16 + split - 1) / split;  // groups of eight outputs of an owner
    auto first = [&](int r) { return (16 * r + split - 1) / split; };
    const uint32_t bias0 = smem_addr(ctl->bias);
    if (PUSH && split > 1) cluster_wait();  // every CTA has started
    {
        const int q = warp & 3;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        const int n = 32 * q + lane;
        const int owner = (n >> 3) * split >> 4;
        const uint32_t push = PUSH && split > 1 ? mapa_shared(recv, static_cast<uint32_t>(owner)) +
                                                      32u * static_cast<uint32_t>(rank * rows * most + (n >> 3) - first(owner)) +
                                                      4u * (n & 7)
                                                : 0u;
        // Sixteen rows of the sums, from row c on.
        auto deliver = [&](int c, const uint32_t (&r)[16]) {
            if (PUSH && split > 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < rows)
                        st_cluster_f32(push + 32u * static_cast<uint32_t>((c + i) * most), __uint_as_float(r[i]));
            } else if (split > 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * 128 + n] = __uint_as_float(r[i]);
            } else {
                // By way of shared memory, a warp its own, from a column a thread
                // to eight adjacent outputs of two rows a thread.
                const uint32_t turn = smem_addr(part) + static_cast<uint32_t>(warp * 2048);
#pragma unroll
                for (int i = 0; i < 16; ++i) st_shared_u32(turn + static_cast<uint32_t>(i * 128 + lane * 4), r[i]);
                __syncwarp();
#pragma unroll 1
                for (int i = lane >> 2; i < min(16, rows - c); i += 8) {
                    const uint32_t at = turn + static_cast<uint32_t>(i * 128 + (lane & 3) * 32);
                    const uint4 lo = ld_shared_v4(at), hi = ld_shared_v4(at + 16);
                    Pair v[4] = {make_pair2(__uint_as_float(lo.x), __uint_as_float(lo.y)),
                                 make_pair2(__uint_as_float(lo.z), __uint_as_float(lo.w)),
                                 make_pair2(__uint_as_float(hi.x), __uint_as_float(hi.y)),
                                 make_pair2(__uint_as_float(hi.z), __uint_as_float(hi.w))};
                    const int d = 32 * q + 8 * (lane & 3);
                    finish_eight<SUMS>(p, b, m0 + c + i, n0 + d, v, bias0 + 4u * d, alpha, beta);
                }
                __syncwarp();
            }
        };
        if constexpr (SUMS) {
            if (warp >= FIRST) {
#pragma unroll
                for (int i = 0; i < ROWS; i += 16) {
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(kept[i + e]);
                    if (row0 + i < rows) deliver(row0 + i, r);
                }
            }
        } else {
            // All eight warps: two share a quarter of the accumulator's lanes and take turns
            // at its rows.
#pragma unroll 1
            for (int c = 16 * (warp >> 2); c < rows; c += 32) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(t_row + static_cast<uint32_t>(c), r);
                tmem_ld_wait();
                if (p.k_blocks == 0) {  // K = 0
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0u;
                }
                deliver(c, r);
            }
            tc_fence_before();
        }
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync_all();
        // CTA `rank` adds the partials of its outputs in rank order, eight
        // adjacent ones a thread.
        const int d0 = PUSH ? first(rank) : 0, count = PUSH ? first(rank + 1) - d0 : 16;
        const int i0 = PUSH ? 0 : rows * rank / split * 16, i1 = PUSH ? rows * count : rows * (rank + 1) / split * 16;
        const uint32_t part_addr = smem_addr(part);
        const uint32_t step = PUSH ? 32u * static_cast<uint32_t>(rows * most) : 0u;
#pragma unroll 1
        for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += THREADS) {
            const int m = i / count, d = d0 + i % count;
            const uint32_t at = PUSH ? recv + 32u * static_cast<uint32_t>(m * most + d - d0) : part_addr + 32u * i;
            Pair v[4] = {};
#pragma unroll 4
            for (int c = 0; c < split; ++c) {
                const uint32_t from = mapa_shared(at + static_cast<uint32_t>(c) * step, static_cast<uint32_t>(PUSH ? rank : c));
                const float4 lo = ld_cluster_f4(from), hi = ld_cluster_f4(from + 16);
                v[0] = add2(v[0], make_pair2(lo.x, lo.y));
                v[1] = add2(v[1], make_pair2(lo.z, lo.w));
                v[2] = add2(v[2], make_pair2(hi.x, hi.y));
                v[3] = add2(v[3], make_pair2(hi.z, hi.w));
            }
            finish_eight<SUMS>(p, b, m0 + m, n0 + 8 * d, v, bias0 + 32u * d, alpha, beta);
        }
    }
    if (!PUSH && split > 1) cluster_sync_all();  // the peers have read this CTA's partials
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
}

// ---------------------------------------------------------------- host side
// The kernels' dynamic shared-memory limit is set once a device.
bool allow_smem(const void* kernel, int slot) {
    static std::mutex mu;
    static bool done[64][8] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!done[dev][slot])
        done[dev][slot] =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem) == cudaSuccess;
    return done[dev][slot];
}

template <int MT, bool SUMS>
int launch(const ProductLaunch& L, int slot, int split, bool two, cudaStream_t stream) {
    if (MT < 64 && L.a_mn) return GEMM_ERR_UNSUPPORTED;  // an MN-major operand comes in chunks of 64
    FewParams p = {};
    constexpr int STAGE = P_TILE_BYTES + MT * PK * 2;
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.k_blocks = static_cast<int>((L.K + PK - 1) / PK);
    p.tiles_m = static_cast<int>((L.M + MT - 1) / MT);
    p.tiles_n = static_cast<int>((L.N + 127) / 128);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * L.batch;
    p.split = split;
    if (tiles * split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    p.tmem_cols = 32;
    while (static_cast<int>(p.tmem_cols) < (SUMS ? 2 : 1) * MT) p.tmem_cols *= 2;
    if (p.tmem_cols > 256) two = false;
    // Two CTAs an SM with half of shared memory each, or a ring as deep as one
    // CTA's room.
    const int budget = (two ? 112 : 226) * 1024;
    // Room for pushed partials: ceil(16/c) groups of eight of a row from each of c CTAs.
    const int recv = MT <= kPush && split > 1 ? static_cast<int>(L.M < MT ? L.M : MT) * (16 + split) * 32 : 0;
    const int stages = (budget - 1024 - static_cast<int>(sizeof(FewCtl)) - recv) / STAGE;
    static_assert(4 * STAGE >= MT * 512, "other partials lie over the ring");
    p.stages = stages < kMaxStages ? stages : kMaxStages;
    p.f_mn = L.b_mn;
    p.t_mn = L.a_mn;
    p.f_whole = p.N - 127;
    p.t_whole = p.M - (MT - 1);
    p.idesc = product_instruction(128, MT, L.bf16, L.b_mn, L.a_mn);
    p.epi = L.epi;
    p.act = L.act;
    p.bf16 = L.out_bf16;
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
    int smem = 1024 + p.stages * STAGE + static_cast<int>(sizeof(FewCtl)) + recv;
    const int least = p.tmem_cols > 256 ? kTmemAloneSmem : kTmemPairedSmem;
    if (smem < least) smem = least;
    if (L.plan) {
        *L.plan = {LINEAR_KERNEL_FEW, MT, split, p.stages, static_cast<int>(tiles * split), smem};
        return GEMM_OK;
    }
    FewMaps maps = {};
    if (L.K > 0 && (!encode_operand(&maps.F, &maps.F_edge, L.B, L.b_mn, L.bf16, L.N, L.K, L.batch, 128) ||
                    !encode_operand(&maps.T, &maps.T_edge, L.A, L.a_mn, L.bf16, L.M, L.K, L.batch, MT)))
        return GEMM_ERR_LAUNCH;
    auto kernel = product_few_kernel<MT, SUMS>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), slot)) return GEMM_ERR_LAUNCH;
    ProductConfig c(tiles * split, split, 32 * kWarps<MT, SUMS>, smem, stream);
    return product_finish(cudaLaunchKernelEx(&c.cfg, kernel, maps, p));
}

// Which kernel, tile and cut of K: the one with the least time by a model in
// microseconds, whose constants were fitted to every choice measured on 82 shapes of
// 1 to 30000 rows (the pairs' K blocks to large shapes alone).  On those its choices
// are 2 % slower than the best one of each on average, 15 % at most (dw 8192 x 512 x
// 512: 16.0 us for 13.9).
//   * few rows: a round of resident CTAs takes each one's K blocks and an
//     epilogue that grows with the rows, and a cut K the partials' way through
//     distributed shared memory.  A K block takes its products and copies, more where
//     two CTAs share an SM, or what the SM's port to L2 takes for its bytes (156 GB/s).
//   * pairs: a round takes its K blocks and the part of an epilogue that does not run
//     under products, the launch another.
struct Choice {
    int mt = 0;  // 0: the pair kernel
    int bn = 256;  // its tiles' width
    int split = 1;
    bool two = false;  // two CTAs an SM
};

// Whether a K cut in `split` leaves a CTA more blocks than one accumulator sums.
bool takes_sums(const ProductLaunch& L, int split) {
    const int64_t kb = (L.K + PK - 1) / PK;
    return L.epi == EPI_F32 && (kb + split - 1) / split > kProductChunk;
}

bool choose(const ProductLaunch& L, Choice* best) {
    // CTAs that run at once, one an SM or two.  (A cluster lies within a GPC: two CTAs
    // an SM take half of its SMs.)
    int resident[2][9];
    if (!product_resident_ctas(resident[0])) return false;
    for (int c = 0; c <= 8; ++c) resident[1][c] = 2 * resident[0][c % 2 == 0 ? c / 2 : c];
    const int64_t kb = (L.K + PK - 1) / PK;
    if (kb == 0) {  // no operands to read: the epilogue alone
        best->mt = 128;
        return true;
    }
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t tm = up(L.M, 256);
    const int64_t units = product_resident_pairs();
    if (units <= 0) return false;
    // Memory's rate bounds every choice alike but for what lies beside the bytes.
    const double bytes = L.batch * (2.0 * static_cast<double>(L.M + L.N) * L.K +
                                    (L.epi == EPI_F32 ? 4.0 : 2.0) * static_cast<double>(L.M) * L.N);
    auto bounded = [&](double us, double rate) { return 0.05 * us + (us > 3.0 + bytes / rate ? us : 3.0 + bytes / rate); };
    double least = 1e30;
    // Microseconds of a K block by the tile's width: 256, 224, 192.  (An MN-major B's
    // narrower tiles do not start on whole 128-byte lines.)
    const double kBlock[3] = {0.288, L.b_mn ? 0.285 : 0.262, L.b_mn ? 0.262 : 0.236};
    for (int w = 0; w < (L.symmetric ? 1 : 3); ++w) {
        const int bn = 256 - 32 * w;
        const int64_t tn = up(L.N, bn);
        const int64_t pairs = (L.symmetric ? tm * (tm + 1) / 2 : tm * tn) * L.batch;
        const double end = 0.9 * bn / 256 + (L.symmetric ? 1.2 : 0.0);  // (a mirror image is stored too)
        const double us = bounded(4.0 + end + static_cast<double>(up(pairs, units)) * (kBlock[w] * kb + end), 5.1e6);
        if (us < least) {
            least = us;
            best->bn = bn;
        }
    }
    const int mt0 = L.a_mn ? 64 : 16;
    for (int mt = mt0; mt <= 256 && (mt == mt0 || mt < 2 * L.M); mt *= 2) {
        const int64_t tiles = up(L.M, mt) * up(L.N, 128) * L.batch;
        for (int c = 1; c <= 8 && c <= kb; ++c) {
            if (resident[0][c] <= 0) continue;
            const int64_t accs = takes_sums(L, c) ? 2 : 1;
            const int64_t ctas = tiles * c;
            if (ctas > 0x7fffffff) continue;
            const double rows = static_cast<double>(mt < L.M ? mt : L.M);
            for (int t = 0; t <= (mt <= kTwo && accs * mt <= 256 ? 1 : 0); ++t) {
                const bool shared = t && ctas > resident[0][c];  // two CTAs an SM, not one
                const double slower = shared ? 1.18 : 1.0;
                const double block = 0.199 + 0.00042 * mt + (t && !shared ? 0.03 : 0.0);
                const double port = (shared ? 2.0 : 1.0) * (P_TILE_BYTES + PK * 2.0 * mt) / 156e3;
                const double rounds = static_cast<double>(up(ctas, resident[t][c]));
                double us = (t ? 0.53 : 0.67) +
                            rounds * (up(kb, c) * (slower * block > port ? slower * block : port) +
                                      slower * (c > 1 ? 3.1 + 0.0427 * rows : 2.36 + 0.0168 * rows));
                if (c > 1) us += (shared ? 0.157 : 0.1) * c - 0.0088 * rows - 0.46;
                us = bounded(us, 5.75e6);
                if (us < least) {
                    least = us;
                    best->mt = mt;
                    best->split = c;
                    best->two = t == 1;
                }
            }
        }
    }
    return true;
}

}  // namespace

bool product_resident_ctas(int (&out)[9]) {
    static std::mutex mu;
    static bool known[64] = {};
    static int n[64][9] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const void* kernel = reinterpret_cast<const void*>(product_few_kernel<128, false>);
    if (!allow_smem(kernel, 3)) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!known[dev]) {
        for (int c = 1; c <= 8; ++c) {
            ProductConfig cfg(c, c, 32 * kWarps<128, false>, 200 * 1024, nullptr);
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

int product_few_launch(const ProductLaunch& L, int mt, int split, bool two, cudaStream_t stream) {
    if (takes_sums(L, split)) {  // (an fp32 result's tiles have 64 rows at least)
        switch (mt) {
            case 64: return launch<64, true>(L, 5, split, two, stream);
            case 128: return launch<128, true>(L, 6, split, two, stream);
            default: return launch<256, true>(L, 7, split, two, stream);
        }
    }
    switch (mt) {
        case 16: return launch<16, false>(L, 0, split, two, stream);
        case 32: return launch<32, false>(L, 1, split, two, stream);
        case 64: return launch<64, false>(L, 2, split, two, stream);
        case 128: return launch<128, false>(L, 3, split, two, stream);
        default: return launch<256, false>(L, 4, split, two, stream);
    }
}

int product_launch(const ProductLaunch& L, cudaStream_t stream) {
    Choice c;
    if (!choose(L, &c)) return GEMM_ERR_CUDA;
    return c.mt ? product_few_launch(L, c.mt, c.split, c.two, stream) : product_pair_launch(L, c.bn, stream);
}

int product_few_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_product_few_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_product_few_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace ssp
