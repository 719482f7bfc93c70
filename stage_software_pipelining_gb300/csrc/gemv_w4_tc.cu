// gemv_w4_tc.cu -- the 4-bit product for more than 16 rows of x, on tcgen05.
//
// Taken where the warp-level products of gemv_w4.cu fill too much of the tensor
// pipe: 32 x 8192 x 28672 (groups of 128, fp16) takes 40 us here and 64 us with
// mma.sync, of which 25 us are the 16 x 8 x 16 products alone; 16 x 8192 x 8192
// takes 15 us here and 14 us there.  The weights' bytes alone are 18 us of the
// first; what bounds it is the instructions that unpack (two thirds of the issue
// slots of an SM with two CTAs) and a chunk's way through the warps.
//
// A CTA takes 128 weight rows (the M side of the product; the rows of x are its
// N side) and a part of K, and its warps hand it on:
//   * one copies blocks of the packed weights and of x into a ring of
//     shared-memory stages (tensor copies, 128 of K a stage);
//   * four or eight unpack: a thread owns a weight row, turns its nibbles into exact
//     16-bit w - zero and stores them to tensor memory, from where tcgen05.mma
//     takes its A operand: they never go back to shared memory;
//   * one issues the products; a group's sums go to TMEM columns of their own;
//   * four add: the row's thread reads its sums back, scales them in fp32 and
//     adds (no weight is rounded, whatever its scale).
// K is also cut over the CTAs of a cluster, whose partials are added in rank
// order through distributed shared memory.
#include <type_traits>

#include "gemv_w4.cuh"

namespace ssp {
namespace {

using namespace w4;

constexpr int R = 128;              // weight rows of a tile: the lanes of TMEM
constexpr int NC = 32;              // rows of x a tile: the product's N
constexpr int NB = 2;               // chunks in flight between unpacking and products
constexpr int KT = 128;             // K of a stage: 64 bytes of a row's nibbles
constexpr int W_BYTES = R * KT / 2; // 8 KB
constexpr int ATOM = NC * 128;      // bytes of x's rows by 64 of K
constexpr int X_BYTES = KT / 64 * ATOM;
constexpr int SLOT = W_BYTES + X_BYTES;
constexpr int kStages = 6;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kDCols = 128;    // TMEM columns of the accumulators, after the A operand's 128

// Eight 4-bit weights less their zero point as four pairs (k, k + 1), exact in
// 16 bits, the order in which x lies in memory.  A byte goes into both halves
// and a nibble of it is kept in each, under an exponent as in unpack(): fp16
// keeps the upper one in place and takes a sixteenth of it (12 instructions),
// bf16 needs a shifted copy (13).  zero: from zero_pair().
template <bool BF16>
__device__ __forceinline__ void unpack_adjacent(uint32_t w, uint32_t zero, uint32_t* p) {
    const uint32_t up = w >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const uint32_t v = __byte_perm(w, up, (4 + i) << 8 | i);
            p[i] = u32(__hsub2(b2(and_or(v, 0x000f000fu, 0x43004300u)), b2(zero)));
        } else {
            const uint32_t v = __byte_perm(w, w, i << 8 | i);
            p[i] = u32(__hfma2(h2(and_or(v, 0x00f0000fu, 0x64006400u)), h2(0x2c003c00u), h2(zero)));
        }
    }
}
// bf16 128 + z twice; fp16 -(1024 + z) below -(64 + z).
template <bool BF16>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
    return BF16 ? z * 0x00010001u + 0x43004300u : z * 0x00100001u + 0xd400e400u;
}

template <int GROUP>
struct Geo {
    // K of a chunk, the unit handed from the unpacking warps to the MMA warp: NB
    // of them in the A operand's TMEM columns, their groups' sums in D's.
    static constexpr int KC = NB * (128 / GROUP) * NC <= static_cast<int>(kDCols) ? 128 : 64;
    static constexpr int SUB = KC / GROUP;  // groups of a chunk
    static constexpr int CPS = KT / KC;     // chunks of a stage
    // Sets of four unpacking warps, which take chunks in turn.  With groups of 128
    // a second one pays: 20 x 28672 x 8192 takes 38.4 us against 42.3 (24 x 4096^2
    // 8.0 against 7.9).  With groups of 32 it does not, 66.9 against 62.0: the
    // adding warps are the slower ones, and are left fewer registers.
    static constexpr int SETS = GROUP == 128 ? 2 : 1;
    static constexpr int kThreads = 64 + 128 * SETS + 128;  // TMA warp, MMA warp, unpacking, adding
    static constexpr int kAdd = 2 + 4 * SETS;               // first adding warp
    static constexpr int LD = SETS == 1 ? NC : NC / 2;      // sums an adding thread reads at once
    static constexpr int RUN = SETS == 1 ? 8 : 4;           // scales or zero points of a row fetched at once
    static_assert(NB % SETS == 0 && kStages % SETS == 0 && (SETS == 1 || CPS == 1) && SETS * SUB <= RUN, "the sets' turns");
    static_assert(KC >= GROUP && NB * SUB * NC <= static_cast<int>(kDCols), "TMEM");
};

struct Ctl {
    // full, empty [kStages]; A in TMEM, products made, sums read [NB]; drain
    unsigned long long bar[2 * kStages + 3 * NB + 1];
    uint32_t tmem_base;
    int abort;
};
constexpr int kUsed = 1024 + kStages * SLOT + static_cast<int>(sizeof(Ctl));
constexpr int kSmem = kUsed > kTmemPairedSmem ? kUsed : kTmemPairedSmem;
static_assert(2 * (kSmem + kCtaSmem) <= kSmSmem && 2 * kTmemCols <= 512, "two CTAs an SM");
static_assert(NC * R * 4 <= kStages * SLOT, "the partials lie over the ring");

template <bool BF16, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(Geo<GROUP>::kThreads, 2)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int SUB = Geo<GROUP>::SUB, KC = Geo<GROUP>::KC, CPS = Geo<GROUP>::CPS;
    constexpr int S = kStages, SETS = Geo<GROUP>::SETS, kAdd = Geo<GROUP>::kAdd, LD = Geo<GROUP>::LD;
    constexpr int kThreads = Geo<GROUP>::kThreads, RUN = Geo<GROUP>::RUN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* x_ring = smem + S * W_BYTES;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + S * SLOT);
    float* part = reinterpret_cast<float*>(smem);  // [NC][R], over the ring once it is read

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cl = static_cast<int>(blockIdx.x) / split;
    const int m0 = (cl % p.tiles_m) * NC, n0 = (cl / p.tiles_m) * R;
    const int k0 = static_cast<int>(static_cast<long long>(p.blocks) * rank / split);
    const int k1 = static_cast<int>(static_cast<long long>(p.blocks) * (rank + 1) / split);
    const uint32_t bar0 = smem_addr(&ctl->bar[0]);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto afull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };           // A chunk b is in TMEM
    auto done_bar = [&](int b) { return bar0 + 8u * (2 * S + NB + b); };       // its products are made
    auto dread_bar = [&](int b) { return bar0 + 8u * (2 * S + 2 * NB + b); };  // its sums are read
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 3 * NB);
    volatile int* abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 5);  // a set of unpacking warps and the products that read x
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(afull_bar(b), 4);
            mbar_init(done_bar(b), 1);
            mbar_init(dread_bar(b), 4);
        }
        mbar_init(drain_bar, 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&ctl->tmem_base), kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_a = ctl->tmem_base, tmem_d = tmem_a + 128u;
    griddep_launch_dependents();
    griddep_wait();

    float acc[NC] = {};
    int issued = 0;  // thread 0: stages
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int kb = k0; kb < k1; ++kb, ++issued) {
                if (!wait_for(empty_bar(s), ph ^ 1u, abort_flag, p.wait_limit_ns)) break;
                if (!(issued == p.withhold && blockIdx.x == 0)) {
                    mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(W_BYTES + (KT / 64) * p.x_rows * 128));
                    tma_load_2d(smem_addr(smem + s * W_BYTES), &tmW, full_bar(s), kb * (KT / 2), n0);
#pragma unroll
                    for (int a = 0; a < KT / 64; ++a)
                        tma_load_2d(smem_addr(x_ring + s * X_BYTES + a * ATOM), &tmX, full_bar(s), kb * KT + a * 64,
                                    m0);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        int s = 0, i = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int kb = k0; ok && kb < k1; ++kb) {
            const Wait full(full_bar(s), ph);  // x is there
            const uint64_t x_desc = k_major_desc(smem_addr(x_ring + s * X_BYTES));
            for (int ch = 0; ch < CPS; ++ch, ++i) {
                const int b = i % NB;
                const uint32_t bp = static_cast<uint32_t>(i / NB) & 1u;
                const Wait dread(dread_bar(b), bp ^ 1u), afull(afull_bar(b), bp);
                if ((ch == 0 && !full.done(abort_flag, p.wait_limit_ns)) ||
                    !dread.done(abort_flag, p.wait_limit_ns) || !afull.done(abort_flag, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // One election a chunk: electing a lane for every product costs
                // about 108 clocks each, these take 29 (N = 16) to 35 (N = 32).
                const uint64_t xd = x_desc + static_cast<uint32_t>((ch * KC / 64 * ATOM + ch * KC % 64 * 2) / 16);
                const uint32_t at = tmem_a + static_cast<uint32_t>(b * (KC / 2));
                const uint32_t dt = tmem_d + static_cast<uint32_t>(b * SUB * NC);
                if (elect_one_sync()) {
#pragma unroll
                    for (int kk = 0; kk < KC / 16; ++kk)
                        umma_f16_ts(dt + kk * 16 / GROUP * NC, at + kk * 8,
                                    xd + static_cast<uint32_t>((kk * 16 / 64 * ATOM + kk * 16 % 64 * 2) / 16), p.idesc,
                                    kk * 16 % GROUP != 0);
                    umma_commit(done_bar(b));
                    if (ch == CPS - 1) umma_commit(empty_bar(s));
                }
                __syncwarp();
            }
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
        // Every product this warp issued ends before TMEM is freed.
        if (elect_one_sync()) umma_commit(drain_bar);
        __syncwarp();
        drain_wait(drain_bar, 0u, p.wait_limit_ns);
        tc_fence_after();
        tc_fence_before();
    } else if (warp < kAdd) {
        const int q = warp & 3;         // TMEM lane quarter
        const int r = 32 * q + lane;    // this thread's weight row of the tile
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        // Rows past N read the last row's zero points; their results are not stored.
        const uint8_t* zp = ZEROS ? p.zeros + static_cast<long long>(min(n0 + r, p.N - 1)) * p.ldz : nullptr;
        const int g0 = k0 * (KT / GROUP), chunks = (k1 - k0) * CPS;
        const int set = SETS == 1 ? 0 : (warp - 2) >> 2;
        // This row's zero points, RUN groups at a time and a run ahead: a load a
        // group would touch 32 lines for 32 values.
        uint32_t z_now[RUN / 4] = {}, z_next[RUN / 4] = {};
        auto fetch = [&](int run) {  // into z_next; 0 past the last group
            if constexpr (ZEROS) {
                const int gi = RUN * run;
                if (gi + RUN <= p.groups && p.z_vec) {
#pragma unroll
                    for (int h = 0; h < RUN / 4; ++h) z_next[h] = __ldg(reinterpret_cast<const uint32_t*>(zp + gi) + h);
                } else {
#pragma unroll
                    for (int h = 0; h < RUN / 4; ++h) {
                        z_next[h] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (gi + 4 * h + e < p.groups) z_next[h] |= static_cast<uint32_t>(zp[gi + 4 * h + e]) << (8 * e);
                    }
                }
            }
        };
        auto zero_at = [&](int gi) -> uint32_t {
            return (RUN == 8 && gi & 4 ? z_now[RUN / 4 - 1] : z_now[0]) >> (8 * (gi & 3)) & 0xffu;
        };
        int run = (g0 + set * SUB) / RUN - 1;
        fetch(run + 1);
        int s = set;
        uint32_t ph = 0;
        for (int i = set; i < chunks; i += SETS) {
            const int ch = i % CPS, b = i % NB;
            const Wait full(full_bar(s), ph), done(done_bar(b), (static_cast<uint32_t>(i / NB) & 1u) ^ 1u);
            const int gi = g0 + i * SUB;
            if (ZEROS && gi / RUN != run) {  // at most one run on: a turn is up to four groups
                run = gi / RUN;
#pragma unroll
                for (int h = 0; h < RUN / 4; ++h) z_now[h] = z_next[h];
                fetch(run + 1);
            }
            uint32_t zero[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) zero[u] = zero_pair<BF16>(ZEROS ? zero_at(gi + u) : 8u);
            const uint32_t w_at = smem_addr(smem + s * W_BYTES) + static_cast<uint32_t>(r * 64);
            if (!full.done(abort_flag, p.wait_limit_ns)) break;
            bool ok = true;
#pragma unroll
            for (int j = 0; j < KC / 32; ++j) {
                const uint4 w = ld_shared_v4(w_at + static_cast<uint32_t>(((ch * (KC / 32) + j) ^ ((r >> 1) & 3)) * 16));
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                uint32_t a[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack_adjacent<BF16>(words[e], zero[j * 32 / GROUP], &a[4 * e]);
                if (j == 0) {  // the products of chunk i - NB have read this part of A
                    ok = done.done(abort_flag, p.wait_limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                }
                tmem_st_32x32b_x16(tmem_a + lanes + static_cast<uint32_t>(b * (KC / 2) + j * 16), a);
            }
            if (!ok) break;
            if (ch == CPS - 1) {  // the stage's weights are read
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_bar(s));
                s += SETS;
                if (s >= S) {
                    s -= S;
                    ph ^= 1u;
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(afull_bar(b));
        }
    } else {
        const int q = warp & 3;
        const int r = 32 * q + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        const uint16_t* sp =
            static_cast<const uint16_t*>(p.scales) + static_cast<long long>(min(n0 + r, p.N - 1)) * p.lds;
        const int g0 = k0 * (KT / GROUP);
        uint32_t s_now[RUN / 2] = {}, s_next[RUN / 2];  // scales, by runs as the zero points
        auto fetch = [&](int run) {
            const int gi = RUN * run;
            if (gi + RUN <= p.groups && p.s_vec) {
                if constexpr (RUN == 8) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp + gi));
                    s_next[0] = v.x, s_next[1] = v.y, s_next[2] = v.z, s_next[3] = v.w;
                } else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp + gi));
                    s_next[0] = v.x, s_next[1] = v.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < RUN / 2; ++e) {
                    const uint32_t lo = gi + 2 * e < p.groups ? sp[gi + 2 * e] : 0u;
                    const uint32_t hi = gi + 2 * e + 1 < p.groups ? sp[gi + 2 * e + 1] : 0u;
                    s_next[e] = lo | hi << 16;
                }
            }
        };
        // Group gi's scale, gi in the run at hand.
        auto scale_of = [&](int gi) -> float {
            uint32_t v = gi & 2 ? s_now[1] : s_now[0];
            if constexpr (RUN == 8) v = gi & 4 ? (gi & 2 ? s_now[3] : s_now[2]) : v;
            const uint16_t h = static_cast<uint16_t>(gi & 1 ? v >> 16 : v);
            return f32_of(*reinterpret_cast<const T*>(&h));
        };
        int run = g0 / RUN - 1;
        fetch(run + 1);
        const int chunks = (k1 - k0) * CPS;
        for (int i = 0; i < chunks; ++i) {
            const int b = i % NB;
            const Wait done(done_bar(b), static_cast<uint32_t>(i / NB) & 1u);
            const int gi = g0 + i * SUB;
            if (gi / RUN != run) {
                run = gi / RUN;
#pragma unroll
                for (int e = 0; e < RUN / 2; ++e) s_now[e] = s_next[e];
                fetch(run + 1);
            }
            float scale[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) scale[u] = scale_of(gi + u);
            if (!done.done(abort_flag, p.wait_limit_ns)) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
                for (int h = 0; h < NC; h += LD) {
                    uint32_t d[LD];
                    const uint32_t at = tmem_d + lanes + static_cast<uint32_t>((b * SUB + u) * NC + h);
                    if constexpr (LD == 32) tmem_ld_32x32b_x32(at, d);
                    else tmem_ld_32x32b_x16(at, d);
                    tmem_ld_wait();
                    if (u == SUB - 1 && h == NC - LD) {  // the sums' columns are free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dread_bar(b));
                    }
#pragma unroll
                    for (int m = 0; m < LD; m += 2) fma2(acc[h + m], acc[h + m + 1], __uint_as_float(d[m]), __uint_as_float(d[m + 1]), scale[u]);
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();  // the ring is read and the products are made
    if (*abort_flag) {
        // Copies that nobody waited for land before the ring is reused.
        if (threadIdx.x == 0)
            for (int j = issued - S > 0 ? issued - S : 0; j < issued; ++j) {
                if (j == p.withhold && blockIdx.x == 0) continue;
                drain_wait(full_bar(j % S), static_cast<uint32_t>((j / S) & 1), p.wait_limit_ns);
            }
        __syncthreads();
    }
    if (warp >= kAdd) {
        const int r = 32 * (warp & 3) + lane;
#pragma unroll
        for (int m = 0; m < NC; ++m) part[m * R + r] = acc[m];
    }
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // CTA `rank` adds the cluster's partials of its share of the outputs, in
    // order, four adjacent ones a thread.
    const int total = min(NC, p.M - m0) * (R / 4);
    const uint32_t part_addr = smem_addr(part);
    for (int i = total * rank / split + static_cast<int>(threadIdx.x); i < total * (rank + 1) / split; i += kThreads) {
        float4 u[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < split)
                u[c] = split == 1 ? *reinterpret_cast<const float4*>(part + 4 * i)
                                  : ld_cluster_f4(mapa_shared(part_addr + 16u * i, static_cast<uint32_t>(c)));
#pragma unroll
        for (int c = 1; c < 8; ++c)
            if (c < split) add4(u[0], u[c]);
        store4<T>(p, m0 + i / (R / 4), n0 + i % (R / 4) * 4, u[0]);
    }
    if (split > 1) cluster_sync_all();  // the peers have read this CTA's partials
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_a, kTmemCols);
    }
}

template <bool BF16, int GROUP, bool ZEROS>
int launch_one(const W4Launch& L, cudaStream_t stream) {
    Params p = params_of(L);
    p.blocks = static_cast<int>((L.K + KT - 1) / KT);
    p.tiles_m = static_cast<int>((L.M + NC - 1) / NC);
    p.x_rows = static_cast<int>(L.M < NC ? L.M : NC);
    p.stages = kStages;
    // Instruction descriptor (kind::f16): D fp32, A and B fp16 (0) or bf16 (1),
    // both K-major, N >> 3 at bits 17..22, M >> 4 at bits 24..28.
    const uint32_t fmt = BF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(NC >> 3) << 17) | (8u << 24);
    auto kernel = w4_tc_kernel<BF16, GROUP, ZEROS>;
    static Residency res;
    int resident[9];
    constexpr int kThreads = Geo<GROUP>::kThreads;
    if (!res.get(reinterpret_cast<const void*>(kernel), kThreads, kSmem, resident)) return GEMM_ERR_LAUNCH;
    // The runtime counts one CTA an SM for a kernel that allocates TMEM; two run
    // (each takes half of TMEM and of shared memory), as the launch bounds say.
    for (int& n : resident) n *= 2;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * ((L.N + R - 1) / R);
    p.split = choose_split(tiles, p.blocks, 4, resident);
    if (L.plan) return planned(L, QUANT_KERNEL_W4_TC, NC, p, tiles, kSmem);
    CUtensorMap tmW, tmX;
    if (!encode_rows(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_64B, L.W, L.N, L.K / 2, L.ldw, KT / 2, R) ||
        !encode_rows(&tmX, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     CU_TENSOR_MAP_SWIZZLE_128B, L.x, L.M, L.K,
                     L.ldx * 2, 64, p.x_rows))
        return GEMM_ERR_LAUNCH;
    return launch(kernel, tmW, tmX, p, tiles, kThreads, kSmem, stream);
}

template <bool BF16, int GROUP>
int launch_zeros(const W4Launch& L, cudaStream_t stream) {
    return L.zeros ? launch_one<BF16, GROUP, true>(L, stream) : launch_one<BF16, GROUP, false>(L, stream);
}

template <int GROUP>
int launch_group(const W4Launch& L, cudaStream_t stream) {
    return L.bf16 ? launch_zeros<true, GROUP>(L, stream) : launch_zeros<false, GROUP>(L, stream);
}

}  // namespace

int w4_launch_tc(const W4Launch& L, cudaStream_t stream) {
    if (L.group == 32) return launch_group<32>(L, stream);
    if (L.group == 64) return launch_group<64>(L, stream);
    return launch_group<128>(L, stream);
}

int w4_tc_read_and_clear_status(GemmDeviceStatus* out) { return w4::read_and_clear_status(out); }

}  // namespace ssp
