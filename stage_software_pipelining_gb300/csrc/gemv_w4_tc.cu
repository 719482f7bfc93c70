// gemv_w4_tc.cu -- the 4-bit product for more than 16 rows of x, on tcgen05.
//
// Taken where the warp-level products of gemv_w4.cu fill too much of the tensor
// pipe: 32 x 8192 x 28672 (groups of 128, fp16) takes 44 us here and 64 us with
// mma.sync, of which 25 us are the 16 x 8 x 16 products alone; 16 x 8192 x 8192
// takes 18 us here and 14 us there.  The weights' bytes alone are 18 us of the
// first; what bounds it is the latency of a chunk's way through the warps.
//
// A CTA takes 128 weight rows (the M side of the product; the rows of x are its
// N side) and a part of K, and its warps hand it on:
//   * one copies blocks of the packed weights and of x into a ring of
//     shared-memory stages (tensor copies, 256 of K a stage);
//   * four unpack: a thread owns a weight row, turns its nibbles into exact
//     16-bit w - zero and stores them to tensor memory, from where tcgen05.mma
//     takes its A operand: they never go back to shared memory, and scale, zero
//     point and result of a row belong to one thread.  These warps also put x
//     into the order the nibbles come out in;
//   * one issues the products.  A group's sums go to TMEM columns of their own;
//     the row's thread reads them back, scales them in fp32 and adds.  No weight
//     is rounded, whatever its scale.
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
constexpr int kThreads = 192;       // TMA warp, MMA warp, four unpacking warps
constexpr int W_BYTES = R * KS / 2; // 16 KB
constexpr int ATOM = NC * 128;      // bytes of x's rows by 64 of K
constexpr int X_BYTES = KS / 64 * ATOM;
constexpr int SLOT = W_BYTES + X_BYTES;
constexpr int kStages = 3;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kDCols = 128;    // TMEM columns of the accumulators, after the A operand's 128

// Shared-memory descriptor of a K-major operand: 128-byte rows, 8-row groups
// 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}

template <int GROUP>
struct Geo {
    // K of a chunk, the unit handed from the unpacking warps to the MMA warp: NB
    // of them in the A operand's TMEM columns, their groups' sums in D's.
    static constexpr int KC = NB * (128 / GROUP) * NC <= static_cast<int>(kDCols) ? 128 : 64;
    static constexpr int SUB = KC / GROUP;  // groups of a chunk
    static constexpr int CPS = KS / KC;     // chunks of a stage
    static_assert(KC >= GROUP && NB * SUB * NC <= static_cast<int>(kDCols), "TMEM");
};

struct Ctl {
    // full, empty [kStages]; A in TMEM, products made [NB]; drain
    unsigned long long bar[2 * kStages + 2 * NB + 1];
    uint32_t tmem_base;
    int abort;
};
constexpr int kSmem = 1024 + kStages * SLOT + static_cast<int>(sizeof(Ctl));
static_assert(NC * R * 4 <= kStages * SLOT, "the partials lie over the ring");

template <bool BF16, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 2)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int SUB = Geo<GROUP>::SUB, KC = Geo<GROUP>::KC, CPS = Geo<GROUP>::CPS;
    constexpr int S = kStages;
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
    auto afull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };       // A chunk b is in TMEM
    auto done_bar = [&](int b) { return bar0 + 8u * (2 * S + NB + b); };  // its products are made
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * NB);
    volatile int* abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 5);  // the unpacking warps and the products that read x
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(afull_bar(b), 4);
            mbar_init(done_bar(b), 1);
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
                    mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(W_BYTES + (KS / 64) * p.x_rows * 128));
                    tma_load_2d(smem_addr(smem + s * W_BYTES), &tmW, full_bar(s), kb * (KS / 2), n0);
#pragma unroll
                    for (int a = 0; a < KS / 64; ++a)
                        tma_load_2d(smem_addr(x_ring + s * X_BYTES + a * ATOM), &tmX, full_bar(s), kb * KS + a * 64,
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
            if (!warp_wait(full_bar(s), ph, abort_flag, p.wait_limit_ns)) break;
            const uint64_t x_desc = smem_desc(smem_addr(x_ring + s * X_BYTES));
            for (int ch = 0; ch < CPS; ++ch, ++i) {
                const int b = i % NB;
                if (!warp_wait(afull_bar(b), static_cast<uint32_t>(i / NB) & 1u, abort_flag, p.wait_limit_ns)) {
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
    } else {
        const int q = warp & 3;         // TMEM lane quarter
        const int r = 32 * q + lane;    // this thread's weight row of the tile
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        // Rows past N read the last row's scales; their results are not stored.
        const long long n = min(n0 + r, p.N - 1);
        const uint16_t* sp = static_cast<const uint16_t*>(p.scales) + n * p.lds;
        const uint8_t* zp = ZEROS ? p.zeros + n * p.ldz : nullptr;
        const int g0 = k0 * (KS / GROUP), chunks = (k1 - k0) * CPS;
        // This row's scales and zero points, eight groups (an octet) at a time
        // and one octet ahead: a load a group would touch 32 lines for 32 values.
        uint32_t s_now[4], s_next[4], z_now[2] = {}, z_next[2] = {};
        auto fetch = [&](int octet) {  // into s_next, z_next; 0 past the last group
            const int gi = 8 * octet;
            const bool whole = gi + 8 <= p.groups;
            if (whole && p.s_vec) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp + gi));
                s_next[0] = v.x, s_next[1] = v.y, s_next[2] = v.z, s_next[3] = v.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = gi + 2 * e < p.groups ? sp[gi + 2 * e] : 0u;
                    const uint32_t hi = gi + 2 * e + 1 < p.groups ? sp[gi + 2 * e + 1] : 0u;
                    s_next[e] = lo | hi << 16;
                }
            }
            if constexpr (ZEROS) {
                if (whole && p.z_vec) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(zp + gi));
                    z_next[0] = v.x, z_next[1] = v.y;
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        z_next[h] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (gi + 4 * h + e < p.groups) z_next[h] |= static_cast<uint32_t>(zp[gi + 4 * h + e]) << (8 * e);
                    }
                }
            }
        };
        // Group gi's scale and zero point, gi in the octet at hand.
        auto scale_of = [&](int gi) -> float {
            const uint32_t v = gi & 4 ? (gi & 2 ? s_now[3] : s_now[2]) : (gi & 2 ? s_now[1] : s_now[0]);
            const uint16_t h = static_cast<uint16_t>(gi & 1 ? v >> 16 : v);
            return f32_of(*reinterpret_cast<const T*>(&h));
        };
        auto zero_at = [&](int gi) -> uint32_t { return (gi & 4 ? z_now[1] : z_now[0]) >> (8 * (gi & 3)) & 0xffu; };
        // Adds chunk i's sums, scaled; false after an abort.
        auto add_chunk = [&](int i, const float (&scale)[SUB]) -> bool {
            const int b = i % NB;
            if (!warp_wait(done_bar(b), static_cast<uint32_t>(i / NB) & 1u, abort_flag, p.wait_limit_ns)) return false;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t d[NC];
                tmem_ld_32x32b_x32(tmem_d + lanes + static_cast<uint32_t>((b * SUB + u) * NC), d);
                tmem_ld_wait();
#pragma unroll
                for (int m = 0; m < NC; ++m) acc[m] = fmaf(scale[u], __uint_as_float(d[m]), acc[m]);
            }
            return true;
        };
        int octet = g0 / 8 - 1;
        fetch(octet + 1);
        float prev[SUB] = {};
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        int i = 0;
        for (; i < chunks; ++i) {
            const int ch = i % CPS, b = i % NB;
            if (ch == 0 && !(ok = warp_wait(full_bar(s), ph, abort_flag, p.wait_limit_ns))) break;
            const int gi = g0 + i * SUB;
            if (gi / 8 != octet) {  // at most one octet on: a chunk has up to four groups
                octet = gi / 8;
#pragma unroll
                for (int e = 0; e < 4; ++e) s_now[e] = s_next[e];
                z_now[0] = z_next[0], z_now[1] = z_next[1];
                fetch(octet + 1);
            }
            float scale[SUB];
            uint32_t z0[SUB], z16[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                scale[u] = scale_of(gi + u);
                z0[u] = zero_of<BF16>(ZEROS ? zero_at(gi + u) : 8u);
                z16[u] = zero16_of<BF16>(z0[u]);
            }
            // The chunk's x, 16 bytes (eight k) a thread at a time, into the order
            // the nibbles come out in: k, k + 4 of each half side by side.
#pragma unroll
            for (int e = 0; e < KC / 64 * (NC / 16); ++e) {
                const int row = r / 8 + 16 * (e % (NC / 16));
                const uint32_t at = smem_addr(x_ring + s * X_BYTES) +
                                    static_cast<uint32_t>((ch * (KC / 64) + e / (NC / 16)) * ATOM + row * 128 + r % 8 * 16);
                if (row < p.x_rows) {
                    const uint4 v = ld_shared_v4(at);
                    st_shared_v4(at, make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                                __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)));
                }
            }
            fence_proxy_async_shared();  // the products read it
            const uint32_t w_at = smem_addr(smem + s * W_BYTES) + static_cast<uint32_t>(r * 128);
#pragma unroll
            for (int j = 0; j < KC / 32; ++j) {
                const uint4 w = ld_shared_v4(w_at + static_cast<uint32_t>(((ch * (KC / 32) + j) ^ (r & 7)) * 16));
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                uint32_t a[16];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    unpack<BF16>(words[e], z0[j * 32 / GROUP], z16[j * 32 / GROUP],
                                 *reinterpret_cast<uint32_t(*)[4]>(&a[4 * e]));
                tmem_st_32x32b_x16(tmem_a + lanes + static_cast<uint32_t>(b * (KC / 2) + j * 16), a);
            }
            if (ch == CPS - 1) {  // the stage's weights are read
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_bar(s));
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(afull_bar(b));
            // Meanwhile the previous chunk's sums.  The next chunk that this one
            // leaves room for (NB on) is stored after this wait, so its products
            // neither meet A half read nor overwrite sums that are still needed.
            if (i > 0 && !(ok = add_chunk(i - 1, prev))) break;
#pragma unroll
            for (int u = 0; u < SUB; ++u) prev[u] = scale[u];
        }
        if (ok && chunks > 0) add_chunk(chunks - 1, prev);
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
    if (warp >= 2) {
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
    if (!res.get(reinterpret_cast<const void*>(kernel), kThreads, kSmem, resident)) return GEMM_ERR_LAUNCH;
    // The runtime counts one CTA an SM for a kernel that allocates TMEM; two run
    // (each takes half of TMEM and of shared memory), as the launch bounds say.
    for (int& n : resident) n *= 2;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * ((L.N + R - 1) / R);
    p.split = choose_split(tiles, p.blocks, 2, resident);
    CUtensorMap tmW, tmX;
    if (!encode_rows(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.W, L.N, L.K / 2, L.ldw, KS / 2, R) ||
        !encode_rows(&tmX, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, L.x, L.M, L.K,
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
