// gemv_w4.cu -- C[i,j] = sum_groups scales[j,g] * sum_{k in g} x[i,k] * (w[j,k] - zeros[j,g])
// with 4-bit weights w, for up to 16 rows of x and for more where the weights are
// few, and the kernel that makes such weights.  (Else: gemv_w4_tc.cu.)
//
// w4_kernel is bound by reading the weights.  A warp of the CTA copies blocks
// of them (64 rows by 256 of K) and of x through a ring of shared-memory stages
// with tensor copies; eight warps turn the nibbles into 16-bit values in
// registers and multiply them with mma.sync, weights as the 16-row operand and
// up to 8 NT rows of x as the columns.  The sums of a group are scaled in fp32
// once they are complete, so that no weight is rounded.  K is also cut over the
// CTAs of a cluster, whose partials are added in order through distributed
// shared memory.
#include <cfloat>
#include <type_traits>

#include "gemv_w4.cuh"

namespace ssp {
namespace {

using namespace w4;

// D = A B + C of 16 x 8 x 16 on one warp, fp32 accumulation.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Geometry of a CTA: CW consuming warps and one that issues copies.  A
// consuming warp takes 32 weight rows of a stage; stages go to the WK groups
// of warps in turn.  Two CTAs an SM.
constexpr int WK = 4;
constexpr int WR = 2;
constexpr int CW = WK * WR;
constexpr int R = 32 * WR;          // weight rows of a tile
constexpr int kThreads = 32 * (CW + 1);
constexpr int kBudget = 100 * 1024; // dynamic shared memory
constexpr int kLeast = 77 * 1024;   // a third CTA does not fit: see launch_one
constexpr int W_BYTES = R * KS / 2;
constexpr int PITCH = R + 4;        // of a partial's rows: no bank conflicts when written
constexpr int QUADS = R / 4;        // of a row's outputs
constexpr int kRecvRow = (QUADS + 8) * 16;  // bytes for a row's partials: at most ceil(QUADS/c) from each of c <= 8

// LONE: a single row of x leaves seven of the eight columns of the product
// empty.  They hold other groups: column j sees x only in the K of the j-th of
// eight running groups and zeros elsewhere, so that eight groups accumulate
// side by side and are scaled together, each by the lane that holds its column,
// where otherwise all four lanes of a row scale the same group.  Taken for
// groups of 32 and 64: 1 x 8192 x 28672 with zero points takes 37.2 us (fp16,
// groups of 32) and 30.2 (64) against 40.5 and 31.3 without; with groups of 128
// 30.7 against 29.6.
template <bool BF16, int NT, bool LONE, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 2)
    w4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int MT = 8 * NT;
    constexpr int GPS = KS / GROUP;      // groups of a stage
    static_assert(!LONE || (NT == 1 && GPS >= 4), "a lane's two groups are of one stage");
    constexpr int LG = (GPS + 3) / 4;    // values a lane loads where four lanes share a row's groups
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ unsigned long long bars[3 * kMaxStages];
    __shared__ uint4 no_x[LONE ? 32 : 1];  // zeros, as long as one row of x in a stage
    __shared__ int abort_word;
    const int S = p.stages;
    const int x_rows = LONE ? 1 : p.x_rows;
    const int x_bytes = x_rows * KS * 2;
    const int x_slot = (x_bytes + 127) & ~127;
    uint8_t* x_ring = smem + S * W_BYTES;
    float* part = reinterpret_cast<float*>(smem);  // over the ring once it is read
    const uint32_t recv = smem_addr(x_ring + S * x_slot);  // the cluster's partials of this CTA's outputs

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cl = static_cast<int>(blockIdx.x) / split;
    const int m0 = (cl % p.tiles_m) * MT, n0 = (cl / p.tiles_m) * R;
    const int k0 = static_cast<int>(static_cast<long long>(p.blocks) * rank / split);
    const int k1 = static_cast<int>(static_cast<long long>(p.blocks) * (rank + 1) / split);
    const uint32_t bar0 = smem_addr(bars);
    // A slot has two full barriers, for its even and odd turns.  A warp waits for
    // every WK-th stage, and the slot's stage before the one it waits for may be
    // another warp's and not have landed yet: the parity of a single barrier
    // could not tell that stage's phase from the one after the next.  With two,
    // the phase before the awaited one belongs to a stage that was read before
    // the last stage this warp took was copied.
    auto full_bar = [&](int s, int turn) { return bar0 + 8u * (2 * s + (turn & 1)); };
    auto full_phase = [](int turn) { return static_cast<uint32_t>(turn >> 1) & 1u; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
    volatile int* abort_flag = &abort_word;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s, 0), 1);
            mbar_init(full_bar(s, 1), 1);
            mbar_init(empty_bar(s), WR);
        }
        abort_word = 0;
        fence_barrier_init();
    }
    if (LONE && threadIdx.x < 32) no_x[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    if (split > 1) cluster_arrive_relaxed();  // this CTA has started: its shared memory may be written to
    griddep_launch_dependents();
    griddep_wait();

    int issued = 0;  // the producing thread's stages
    if (warp == CW) {
        if (lane == 0) {
            int s = 0, turn = 0;
            for (int kb = k0; kb < k1; ++kb, ++issued) {
                if (!wait_for(empty_bar(s), (turn & 1) ^ 1, abort_flag, p.wait_limit_ns)) break;
                if (!(issued == p.withhold && blockIdx.x == 0)) {
                    const uint32_t bar = full_bar(s, turn);
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(W_BYTES + x_bytes));
                    tma_load_2d(smem_addr(smem + s * W_BYTES), &tmW, bar, kb * (KS / 2), n0);
                    tma_load_3d(smem_addr(x_ring + s * x_slot), &tmX, bar, 0, m0, kb * (KS / 32));
                }
                if (++s == S) {
                    s = 0;
                    ++turn;
                }
            }
        }
        __syncwarp();
        __syncthreads();
        if (*abort_flag) {
            // Copies that nobody waited for land before the ring is reused.
            if (lane == 0)
                for (int j = issued - S > 0 ? issued - S : 0; j < issued; ++j) {
                    if (j == p.withhold && blockIdx.x == 0) continue;
                    drain_wait(full_bar(j % S, j / S), full_phase(j / S), p.wait_limit_ns);
                }
            __syncthreads();
        }
    } else {
        const int wr = warp % WR, wk = warp / WR;
        const int g = lane >> 2, c = lane & 3;
        // This lane's four weight rows are 8 i + g of the warp's 32.  Rows past N
        // read the last row's scales; their results are not stored.
        const T* s_tile = static_cast<const T*>(p.scales) + n0 * p.lds;
        const uint8_t* z_tile = ZEROS ? p.zeros + n0 * p.ldz : nullptr;
        uint32_t s_off[4], z_off[4];  // within the tile's rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = min(32 * wr + 8 * i + g, p.N - 1 - n0);
            s_off[i] = static_cast<uint32_t>(n * static_cast<int>(p.lds));
            z_off[i] = ZEROS ? static_cast<uint32_t>(n * static_cast<int>(p.ldz)) : 0u;
        }
        auto scale_at = [&](int i, int kb, int group) -> T {
            const int gi = kb * GPS + group;
            return kb < k1 && gi < p.groups ? s_tile[s_off[i] + static_cast<uint32_t>(gi)] : of_f32<T>(0.0f);
        };
        auto zero_at = [&](int i, int kb, int group) -> uint32_t {
            const int gi = kb * GPS + group;
            return kb < k1 && gi < p.groups ? z_tile[z_off[i] + static_cast<uint32_t>(gi)] : 0u;
        };
        // Scales, a stage ahead: [u] group 4u + c of the stage (a lane a group; the
        // others ask for it).  LONE: [0], [1] the columns 2c and 2c + 1 of this
        // lane, fetched where eight groups begin.
        constexpr int SV = LONE ? 2 : LG;
        T sv[SV][4];
        uint32_t zv[LG][4];  // zero points: [u] group 4u + c of the stage
        const bool pairs = LONE && p.s_vec && p.groups % 2 == 0;  // one load takes a lane's two
        auto fetch_scales = [&](int kb) {
            if (LONE && pairs) {
                const int stage = kb + WK * (2 * c / GPS), gi = stage * GPS + 2 * c % GPS;
                const bool in = stage < k1 && gi < p.groups;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t v = in ? *reinterpret_cast<const uint32_t*>(s_tile + s_off[i] + gi) : 0u;
                    const uint16_t h[2] = {static_cast<uint16_t>(v), static_cast<uint16_t>(v >> 16)};
                    sv[0][i] = *reinterpret_cast<const T*>(&h[0]);
                    sv[SV - 1][i] = *reinterpret_cast<const T*>(&h[1]);
                }
                return;
            }
#pragma unroll
            for (int u = 0; u < SV; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int slot = 2 * c + u;
                    if constexpr (LONE) sv[u][i] = scale_at(i, kb + WK * (slot / GPS), slot % GPS);
                    else sv[u][i] = scale_at(i, kb, min(4 * u + c, GPS - 1));
                }
        };
        auto fetch_zeros = [&](int kb) {
            if constexpr (ZEROS) {
#pragma unroll
                for (int u = 0; u < LG; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) zv[u][i] = zero_at(i, kb, min(4 * u + c, GPS - 1));
            }
        };
        if constexpr (!LONE) fetch_scales(k0 + wk);
        fetch_zeros(k0 + wk);

        float acc[2][NT][4] = {};  // scaled sums (LONE: [.][.][0], [2] of rows g, g + 8)
        float sub[2][NT][4] = {};  // sums of the running groups
        int pos = 0;               // LONE: groups so far
        // This lane's word of 16-byte chunk 0 in a 128-byte swizzled row: chunk j
        // of row r lies at chunk j ^ (r & 7).
        const uint32_t w_row = smem_addr(smem) + static_cast<uint32_t>((32 * wr + g) * 128 + 16 * g + 4 * c);
        uint32_t x_off[NT];
#pragma unroll
        for (int b = 0; b < NT; ++b)
            x_off[b] = smem_addr(x_ring) + static_cast<uint32_t>(min(8 * b + (LONE ? 0 : g), x_rows - 1) * 64 + 16 * c);
        const uint32_t no_x_at = smem_addr(no_x) + 16u * c;
        int s = wk, turn = 0;
        for (int kb = k0 + wk; kb < k1; kb += WK) {
            float scale[SV][4];
            uint32_t zero[LG][4];
            if constexpr (LONE) {
                if (pos == 0) fetch_scales(kb);
            } else {
#pragma unroll
                for (int u = 0; u < SV; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) scale[u][i] = f32_of(sv[u][i]);
            }
#pragma unroll
            for (int u = 0; u < LG; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if constexpr (ZEROS) zero[u][i] = zero_of<BF16>(zv[u][i]);
            if (!warp_wait(full_bar(s, turn), full_phase(turn), abort_flag, p.wait_limit_ns)) break;
            if constexpr (!LONE) fetch_scales(kb + WK);
            fetch_zeros(kb + WK);
            const uint32_t w_at = w_row + static_cast<uint32_t>(s * W_BYTES);
            const uint32_t x_at = static_cast<uint32_t>(s * x_slot);
#pragma unroll
            for (int u = 0; u < GPS; ++u) {  // a group of K
                uint32_t z0[4], z16[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (!ZEROS) z0[i] = zero_of<BF16>(8u);
                    else z0[i] = GPS == 1 ? zero[0][i] : __shfl_sync(0xffffffffu, zero[u / 4][i], u % 4, 4);
                    z16[i] = zero16_of<BF16>(z0[i]);
                }
                const bool mine = !LONE || g == pos + u;
#pragma unroll
                for (int jj = 0; jj < GROUP / 32; ++jj) {  // 32 of K
                    const int j = u * (GROUP / 32) + jj;
                    // x of this lane's column and eight k, re-paired (k, k + 4).
                    uint32_t xb[NT][4];
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        uint32_t at;
                        if constexpr (LONE) at = (mine ? x_at + x_off[b] : no_x_at) + 64u * j;
                        else at = x_at + x_off[b] + static_cast<uint32_t>(j * x_rows * 64);
                        const uint4 v = ld_shared_v4(at);
                        xb[b][0] = __byte_perm(v.x, v.z, 0x5410);
                        xb[b][1] = __byte_perm(v.x, v.z, 0x7632);
                        xb[b][2] = __byte_perm(v.y, v.w, 0x5410);
                        xb[b][3] = __byte_perm(v.y, v.w, 0x7632);
                    }
#pragma unroll
                    for (int a = 0; a < 2; ++a) {  // 16 weight rows
                        uint32_t q[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 2 * a + h;
                            const uint32_t w = ld_shared_u32((w_at ^ static_cast<uint32_t>(16 * j)) +
                                                             static_cast<uint32_t>(8 * i * (KS / 2)));
                            unpack<BF16>(w, z0[i], z16[i], q[h]);
                        }
                        const uint32_t lo[4] = {q[0][0], q[1][0], q[0][1], q[1][1]};
                        const uint32_t hi[4] = {q[0][2], q[1][2], q[0][3], q[1][3]};
#pragma unroll
                        for (int b = 0; b < NT; ++b) {
                            mma16816<BF16>(sub[a][b], lo, xb[b][0], xb[b][1]);
                            mma16816<BF16>(sub[a][b], hi, xb[b][2], xb[b][3]);
                        }
                    }
                }
                if constexpr (!LONE) {  // the group is complete: scale its sums
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 2 * a + h;
                            const float f =
                                GPS == 1 ? scale[0][i] : __shfl_sync(0xffffffffu, scale[u / 4 % SV][i], u % 4, 4);
#pragma unroll
                            for (int b = 0; b < NT; ++b) {
                                fma2(acc[a][b][2 * h], acc[a][b][2 * h + 1], sub[a][b][2 * h], sub[a][b][2 * h + 1], f);
                                sub[a][b][2 * h] = sub[a][b][2 * h + 1] = 0.0f;
                            }
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(s));
            s += WK;
            if (s >= S) {
                s -= S;
                ++turn;
            }
            if constexpr (LONE) {
                pos += GPS;
                if (pos == 8 || kb + WK >= k1) {
                    pos = 0;
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = 2 * a + (e >> 1), u = e & 1;
                            acc[a][0][e & 2] = fmaf(f32_of(sv[u][i]), sub[a][0][e], acc[a][0][e & 2]);
                            sub[a][0][e] = 0.0f;
                        }
                }
            }
        }
        // The ring is read by every warp before partials lie over it.
        __syncthreads();
        if (*abort_flag) __syncthreads();
        float* mine = part + wk * MT * PITCH;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = 32 * wr + 16 * a + 8 * (e >> 1) + g;
                    float v = acc[a][b][e];
                    if constexpr (LONE) {  // the eight columns are in four lanes
                        if (e & 1) continue;
                        v += __shfl_xor_sync(0xffffffffu, v, 1);
                        v += __shfl_xor_sync(0xffffffffu, v, 2);
                        if (c == 0) mine[n] = v;
                    } else {
                        mine[(8 * b + 2 * c + (e & 1)) * PITCH + n] = v;
                    }
                }
    }
    __syncthreads();
    // Sums over the groups of warps, four adjacent outputs a thread.
    const int rows = min(MT, p.M - m0);
    const float4* part4 = reinterpret_cast<const float4*>(part);
    auto own = [&](int i) {
        const int at = (i / QUADS) * (PITCH / 4) + i % QUADS;
        float4 v = part4[at];
#pragma unroll
        for (int k = 1; k < WK; ++k) add4(v, part4[k * MT * (PITCH / 4) + at]);
        return v;
    };
    if (split == 1) {
        for (int i = static_cast<int>(threadIdx.x); i < rows * QUADS; i += kThreads)
            store4<T>(p, m0 + i / QUADS, n0 + i % QUADS * 4, own(i));
        return;
    }
    // Quad d of a row belongs to CTA d * split / QUADS, to whose shared memory
    // every CTA of the cluster writes its share; the owner adds them in rank
    // order.  (Written by their makers, they need no second barrier to outlive
    // their readers.)
    const int most = (QUADS + split - 1) / split;  // quads of an owner
    auto first = [&](int r) { return (QUADS * r + split - 1) / split; };
    cluster_wait();  // every CTA has started
    for (int i = static_cast<int>(threadIdx.x); i < rows * QUADS; i += kThreads) {
        const int m = i / QUADS, d = i % QUADS, owner = d * split / QUADS;
        st_cluster_f4(mapa_shared(recv, static_cast<uint32_t>(owner)) +
                          16u * static_cast<uint32_t>((rank * rows + m) * most + d - first(owner)),
                      own(i));
    }
    __syncwarp();
    cluster_sync_all();
    const int d0 = first(rank), count = first(rank + 1) - d0;
    for (int i = static_cast<int>(threadIdx.x); i < rows * count; i += kThreads) {
        const int m = i / count, d = i % count;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int r = 0; r < split; ++r) {
            const uint4 u = ld_shared_v4(recv + 16u * static_cast<uint32_t>((r * rows + m) * most + d));
            add4(v, make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)));
        }
        store4<T>(p, m0 + m, n0 + 4 * (d0 + d), v);
    }
}

// Eight weights (one 32-bit word) a thread, group/8 threads a group.
template <typename T, typename S>
__global__ void __launch_bounds__(256, 8) w4_quantize_kernel(const W4QuantLaunch p) {
    const long long words = p.K / 8;
    const long long t = blockIdx.x * 256ll + threadIdx.x;
    const bool in = t < p.N * words;
    // Threads past the end repeat the last word, so that whole warps shuffle.
    const long long u = in ? t : p.N * words - 1;
    // (In 32 bits where they do: a 64-bit division costs more than the rest.)
    const long long j = u >> 32 == 0 ? static_cast<uint32_t>(u) / static_cast<uint32_t>(words) : u / words;
    const int k = static_cast<int>(u - j * words) * 8;
    const T* w = static_cast<const T*>(p.w) + j * p.ld + k;
    alignas(16) T raw[8];
    if (reinterpret_cast<uintptr_t>(w) % 16 == 0) {
#pragma unroll
        for (int e = 0; e < 8 * static_cast<int>(sizeof(T)) / 16; ++e)
            reinterpret_cast<uint4*>(raw)[e] = reinterpret_cast<const uint4*>(w)[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = w[e];
    }
    float v[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = f32_of(raw[e]);
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
    for (int o = p.group / 16; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // Weights too large for a scale of 16 bits take the largest one and are limited.
    constexpr float kMostScale = std::is_same<S, __half>::value ? 65504.0f : 3.38953139e38f;
    float range;
    if (!p.zeros) range = fmaxf(hi, -lo) / 7.0f;
    else if (hi - lo <= FLT_MAX) range = (hi - lo) / 15.0f;
    else range = hi / 15.0f - lo / 15.0f;
    const S s16 = of_f32<S>(fminf(range, kMostScale));
    const float s = f32_of(s16);
    // w / s is often half-way between two integers and must not be off by an ulp
    // there: 1/s in two parts, of which the first is below it (8192 x 8192 bf16,
    // groups of 128: 80.6 us, with a division a weight 90 or more), or a division
    // where 1/s may overflow.
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));  // within an ulp
    const float inv = __int_as_float(__float_as_int(r) - 1), rest = fmaf(-s, inv, 1.0f) * inv;
    // The nearest integer of a quotient, within what the limits 0..15 leave of it:
    // the last bits of its sum with 1.5 * 2^23 (rintf and the conversion are four
    // times slower).
    auto nearest = [](float q) { return __float_as_int(fminf(fmaxf(q, -16.0f), 16.0f) + 0x1.8p23f) - 0x4b400000; };
    auto value = [&](float q, int z) { return static_cast<uint32_t>(min(max(nearest(q) + z, 0), 15)); };
    int z = 8;
    uint32_t word = 0;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        auto quotient = [&](float w) { return fmaf(w, inv, w * rest); };
        if (p.zeros) z = min(nearest(quotient(-lo)), 15);
#pragma unroll
        for (int e = 0; e < 8; ++e) word |= value(quotient(v[e]), z) << (4 * e);
    } else {
        auto quotient = [&](float w) { return s > 0.0f ? w / s : 0.0f; };
        if (p.zeros) z = min(nearest(quotient(-lo)), 15);
#pragma unroll 1
        for (int e = 0; e < 8; ++e) word |= value(quotient(f32_of(w[e])), z) << (4 * e);
    }
    if (!in) return;
    uint8_t* out = p.W + j * p.ldw + k / 2;
    if (reinterpret_cast<uintptr_t>(out) % 4 == 0) {
        *reinterpret_cast<uint32_t*>(out) = word;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = static_cast<uint8_t>(word >> (8 * e));
    }
    if (k % p.group == 0) {
        static_cast<S*>(p.scales)[j * p.lds + k / p.group] = s16;
        if (p.zeros) p.zeros[j * p.ldz + k / p.group] = static_cast<uint8_t>(z);
    }
}

// x as K/32 slices of M rows by 32 elements (64 bytes): a box lands slice by
// slice, so that a warp's 16-byte reads of eight rows touch every bank once.
bool encode_x(CUtensorMap* map, const W4Launch& L, int x_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {32, static_cast<cuuint64_t>(L.M), static_cast<cuuint64_t>(L.K / 32)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(L.ldx * 2), 64};
    cuuint32_t box[3] = {32, static_cast<cuuint32_t>(x_rows), KS / 32};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, L.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(L.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int NT, bool LONE, int GROUP, bool ZEROS>
int launch_one(const W4Launch& L, cudaStream_t stream) {
    Params p = params_of(L);
    p.tiles_m = static_cast<int>((L.M + 8 * NT - 1) / (8 * NT));
    p.x_rows = static_cast<int>(L.M < 8 * NT ? L.M : 8 * NT);
    const int slot = W_BYTES + ((p.x_rows * KS * 2 + 127) & ~127);
    const int stages = (kBudget - 1024 - p.x_rows * kRecvRow) / slot;
    p.stages = stages < kMaxStages ? stages : kMaxStages;
    static_assert(WK * 8 * NT * PITCH * 4 <= 5 * W_BYTES && 5 * (W_BYTES + 8 * NT * KS * 2) + 8 * NT * kRecvRow <= kBudget - 1024,
                  "the partials lie over the ring, which has five stages at least");
    auto kernel = w4_kernel<BF16, NT, LONE, GROUP, ZEROS>;
    static Residency res;
    int resident[9];
    if (!res.get(reinterpret_cast<const void*>(kernel), kThreads, kBudget, resident)) return GEMM_ERR_LAUNCH;
    const int64_t tiles = p.tiles_m * ((L.N + R - 1) / R);
    p.split = choose_split(tiles, p.blocks, 2, resident);
    // Two CTAs an SM, as the split counts on, also where registers would let a
    // third in: with three on some SMs and one on others 1 x 8192 x 28672 (bf16,
    // groups of 128) took 42.8 us, with two on each 30.1.
    int smem = 1024 + p.stages * slot + p.x_rows * kRecvRow;
    if (smem < kLeast) smem = kLeast;
    if (L.plan) return planned(L, QUANT_KERNEL_W4_WARP, 8 * NT, p, tiles, smem);
    CUtensorMap tmW, tmX;
    if (!encode_rows(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, L.W, L.N, L.K / 2, L.ldw, KS / 2, R) ||
        !encode_x(&tmX, L, p.x_rows))
        return GEMM_ERR_LAUNCH;
    return launch(kernel, tmW, tmX, p, tiles, kThreads, smem, stream);
}

template <bool BF16, int NT, bool LONE, int GROUP>
int launch_zeros(const W4Launch& L, cudaStream_t stream) {
    return L.zeros ? launch_one<BF16, NT, LONE, GROUP, true>(L, stream)
                   : launch_one<BF16, NT, LONE, GROUP, false>(L, stream);
}

template <int NT, bool LONE, int GROUP>
int launch_type(const W4Launch& L, cudaStream_t stream) {
    return L.bf16 ? launch_zeros<true, NT, LONE, GROUP>(L, stream) : launch_zeros<false, NT, LONE, GROUP>(L, stream);
}

template <int NT>
int launch_group(const W4Launch& L, cudaStream_t stream) {
    const bool lone = NT == 1 && L.M == 1;
    if (L.group == 32) return lone ? launch_type<1, true, 32>(L, stream) : launch_type<NT, false, 32>(L, stream);
    if (L.group == 64) return lone ? launch_type<1, true, 64>(L, stream) : launch_type<NT, false, 64>(L, stream);
    return launch_type<NT, false, 128>(L, stream);
}

template <typename T>
void quantize_of(const W4QuantLaunch& L, unsigned grid, cudaStream_t stream) {
    if (L.scale_bf16) w4_quantize_kernel<T, __nv_bfloat16><<<grid, 256, 0, stream>>>(L);
    else w4_quantize_kernel<T, __half><<<grid, 256, 0, stream>>>(L);
}

}  // namespace

int w4_launch(const W4Launch& L, cudaStream_t stream) {
    if (L.M <= 8) return launch_group<1>(L, stream);
    if (L.M <= 16) return launch_group<2>(L, stream);
    // More rows than a tile's 16: tiles of them side by side read and unpack the
    // weights again each, but start and end sooner than w4_tc_kernel.  Where the
    // GPU is not full that is less: 24 x 128 x 4096 takes 3.5 us against 5.2, 24 x
    // 1024 x 8192 5.8 against 7.9, 24 x 8192 x 1024 5.4 against 6.4; 17 x 8192 x 2048
    // 8.2 against 7.0, 24 x 4096 x 8192 12.9 against 11.1.
    const int64_t tiles_m = (L.M + 15) / 16, tiles = tiles_m * ((L.N + R - 1) / R);
    const int64_t work = tiles_m * L.N * L.K, sms = tc_current_device_sms();
    if ((tiles <= sms && work <= 1 << 25) || (tiles <= 2 * sms && work <= 1 << 24)) return launch_group<2>(L, stream);
    return w4_launch_tc(L, stream);
}

int w4_read_and_clear_status(GemmDeviceStatus* out) {
    GemmDeviceStatus tc;
    int st = w4::read_and_clear_status(out);
    if (st != GEMM_OK) return st;
    st = w4_tc_read_and_clear_status(&tc);
    if (out->code == 0) *out = tc;
    return st;
}

int w4_quantize_launch(const W4QuantLaunch& L, cudaStream_t stream) {
    const int64_t blocks = (L.N * (L.K / 8) + 255) / 256;
    if (blocks > 0x7fffffffll) return GEMM_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (L.dtype == QUANT_F32) quantize_of<float>(L, grid, stream);
    else if (L.dtype == QUANT_F16) quantize_of<__half>(L, grid, stream);
    else quantize_of<__nv_bfloat16>(L, grid, stream);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace ssp
