// gemv_w4.cu -- C[i,j] = sum_groups scales[j,g] * sum_{k in g} x[i,k] * (w[j,k] - zeros[j,g])
// with 4-bit weights w, and the kernel that makes them.
//
// w4_kernel is bound by reading the weights.  A warp of the CTA copies blocks
// of them (128 or 256 rows by 256 or 128 of K) and of x through a ring of
// shared-memory stages with tensor copies; eight warps turn the nibbles into
// 16-bit values in registers and multiply them with mma.sync, weights as the
// 16-row operand and up to 8 NT rows of x as the columns.  (tcgen05 takes its
// operands from shared memory or TMEM: values that were just unpacked in
// registers would have to be written out again, and the products are far
// from a limit here.)  The sums of a group are scaled in fp32 once they are
// complete, so that no weight is rounded.  K is also cut over the CTAs of a
// cluster, whose partials are added in order through distributed shared memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "../../include/quant.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant.h"

namespace ssp {
namespace {

template <typename T>
__device__ __forceinline__ float f32_of(T v);
template <>
__device__ __forceinline__ float f32_of(float v) { return v; }
template <>
__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T of_f32(float v);
template <>
__device__ __forceinline__ __half of_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 of_f32(float v) { return __float2bfloat16_rn(v); }

constexpr int kWarps = 8;                       // consumer warps; one more issues the copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxStages = 8;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

struct W4Params {
    int M, N, K;
    int tiles_m, groups;  // groups of a row
    int blocks;           // K blocks of KS
    int split;            // CTAs of a cluster, each with a part of the K blocks
    int stages, x_rows;   // ring depth; rows of x in a stage
    const void* scales;
    long long lds;
    const uint8_t* zeros;
    long long ldz;
    void* C;
    long long ldc;
};

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

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

// (a & mask) | magic in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
    return r;
}

__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ __nv_bfloat162 b2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
template <typename V>
__device__ __forceinline__ uint32_t u32(V v) { return *reinterpret_cast<uint32_t*>(&v); }

// Eight 4-bit weights less their zero point, as four pairs (k, k + 4), exact in
// 16 bits.  A nibble under the exponent of 2^7 (bf16: 7 mantissa bits) or 2^10
// (fp16) reads as 128 + w or 1024 + w, from which 128 + z or 1024 + z is
// subtracted; an fp16 nibble four places higher reads as 1024 + 16 w, of which
// a sixteenth less 64 + z is one multiply-add and saves the shift.
template <bool BF16>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t zero, uint32_t zero16, uint32_t (&p)[4]) {
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = u32(__hsub2(b2(and_or(w >> (4 * i), 0x000f000fu, 0x43004300u)), b2(zero)));
    } else {
        const __half2 sixteenth = h2(0x2c002c00u);  // 1/16
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = w >> (8 * i);
            p[2 * i] = u32(__hsub2(h2(and_or(v, 0x000f000fu, 0x64006400u)), h2(zero)));
            p[2 * i + 1] = u32(__hfma2(h2(and_or(v, 0x00f000f0u, 0x64006400u)), sixteenth, h2(zero16)));
        }
    }
}

// The zero point as unpack wants it: (128 + z) or (1024 + z) twice, and for
// fp16 -(64 + z) twice.
template <bool BF16>
__device__ __forceinline__ void zero_of(uint32_t z, uint32_t& zero, uint32_t& zero16) {
    if constexpr (BF16) {
        zero = (0x4300u | z) * 0x00010001u;
        zero16 = 0;
    } else {
        zero = (0x6400u | z) * 0x00010001u;
        zero16 = (0xd400u | (z << 4)) * 0x00010001u;  // -(64 + z): 2^6 has 16 steps a unit
    }
}

// Geometry of a CTA for up to 8 NT rows of x: R weight rows (32 a warp) by
// blocks of KS of K (128 a warp).
template <int NT>
struct Geo {
    static constexpr int WK = NT == 4 ? 1 : 2;   // warps along K
    static constexpr int WR = kWarps / WK;       // warps along the weight rows
    static constexpr int R = 32 * WR;
    static constexpr int KS = 128 * WK;
    static constexpr int W_BYTES = R * KS / 2;
    static constexpr int MT = 8 * NT;
    static constexpr int PITCH = R + 4;          // of a partial's rows: no bank conflicts when written
    static constexpr int PART_FLOATS = WK * MT * PITCH;
};

template <bool BF16, int NT, int GROUP>
__global__ void __launch_bounds__(kThreads, 2)
    w4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const W4Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    using Gm = Geo<NT>;
    constexpr int KS = Gm::KS, R = Gm::R;
    constexpr int SUB = 128 / GROUP;        // groups in a warp's 128 of K
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ unsigned long long bars[2 * kMaxStages];
    __shared__ int abort_word;
    const int S = p.stages;
    const int x_bytes = p.x_rows * KS * 2;
    const int x_slot = (x_bytes + 127) & ~127;
    uint8_t* x_ring = smem + S * Gm::W_BYTES;
    float* part = reinterpret_cast<float*>(smem);  // over the ring once it is read

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cl = static_cast<int>(blockIdx.x) / split;
    const int m0 = (cl % p.tiles_m) * Gm::MT, n0 = (cl / p.tiles_m) * R;
    const int k0 = static_cast<int>(static_cast<long long>(p.blocks) * rank / split);
    const int k1 = static_cast<int>(static_cast<long long>(p.blocks) * (rank + 1) / split);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    volatile int* abort_flag = &abort_word;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), kWarps);
        }
        abort_word = 0;
        fence_barrier_init();
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();

    int issued = 0;  // the producing thread's stages
    if (warp == kWarps) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int kb = k0; kb < k1; ++kb, ++issued) {
                if (!wait_for(empty_bar(s), ph ^ 1u, abort_flag)) break;
                mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(Gm::W_BYTES + x_bytes));
                tma_load_2d(smem_addr(smem + s * Gm::W_BYTES), &tmW, full_bar(s), kb * (KS / 2), n0);
                tma_load_3d(smem_addr(x_ring + s * x_slot), &tmX, full_bar(s), 0, m0, kb * (KS / 32));
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else {
        const int wr = warp % Gm::WR, wk = warp / Gm::WR;
        const int g = lane >> 2, c = lane & 3;
        // The scales (and zero points) of this lane's four rows g, g + 8, g + 16,
        // g + 24 of the warp: lane c of a row's four loads group min(c, SUB - 1)
        // of the warp's 128 of K, one block ahead.  Rows past N read the last
        // row's; their results are not stored.
        const T* sp[4];
        const uint8_t* zp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long n = min(n0 + 32 * wr + 8 * i + g, p.N - 1);
            sp[i] = static_cast<const T*>(p.scales) + n * p.lds;
            zp[i] = p.zeros ? p.zeros + n * p.ldz : nullptr;
        }
        T sv[4];
        uint32_t zv[4];
        auto fetch = [&](int kb) {
            const int gi = kb * (KS / GROUP) + wk * SUB + (c < SUB ? c : SUB - 1);
            const bool in = kb < k1 && gi < p.groups;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sv[i] = in ? sp[i][gi] : of_f32<T>(0.0f);
                zv[i] = !p.zeros ? 8u : in ? zp[i][gi] : 0u;
            }
        };
        fetch(k0);
        float acc[2][NT][4] = {};
        int s = 0;
        uint32_t ph = 0;
        // This lane's byte in a 128-byte (64-byte) swizzled row: 16-byte chunk
        // j of row r is at j ^ (r & 7) (j ^ ((r >> 1) & 3)).
        const uint32_t w_row = static_cast<uint32_t>((32 * wr + g) * (KS / 2) + 4 * c);
        for (int kb = k0; kb < k1; ++kb) {
            float scale[4];
            uint32_t zero[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                scale[i] = f32_of(sv[i]);
                zero[i] = zv[i];
            }
            if (!wait_for(full_bar(s), ph, abort_flag)) break;
            fetch(kb + 1);
            const uint32_t w_at = smem_addr(smem + s * Gm::W_BYTES) + w_row;
            const uint32_t x_at = smem_addr(x_ring + s * x_slot);
            float sub[2][NT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 32 of K
                if (j % (GROUP / 32) == 0)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sub[a][b][e] = 0.0f;
                // x of this lane's column (row of x) and eight k, re-paired (k, k + 4).
                uint32_t xb[NT][4];
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    const int m = min(8 * b + g, p.x_rows - 1);
                    const uint4 v = ld_shared_v4(x_at + static_cast<uint32_t>(((wk * 4 + j) * p.x_rows + m) * 64 + 16 * c));
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
                        const int i = 2 * a + h;  // rows 8 i + g of the warp
                        const int chunk = Gm::WK == 2 ? (wk * 4 + j) ^ g : j ^ ((g >> 1) & 3);
                        const uint32_t w = ld_shared_u32(w_at + static_cast<uint32_t>(8 * i * (KS / 2) + 16 * chunk));
                        const uint32_t z = SUB == 1 ? zero[i] : __shfl_sync(0xffffffffu, zero[i], (lane & 28) + j / (GROUP / 32));
                        uint32_t z0, z16;
                        zero_of<BF16>(z, z0, z16);
                        unpack<BF16>(w, z0, z16, q[h]);
                    }
                    const uint32_t lo[4] = {q[0][0], q[1][0], q[0][1], q[1][1]};
                    const uint32_t hi[4] = {q[0][2], q[1][2], q[0][3], q[1][3]};
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        mma16816<BF16>(sub[a][b], lo, xb[b][0], xb[b][1]);
                        mma16816<BF16>(sub[a][b], hi, xb[b][2], xb[b][3]);
                    }
                }
                if (j % (GROUP / 32) == GROUP / 32 - 1) {  // a group is complete: scale its sums
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 2 * a + h;
                            const float f = SUB == 1 ? scale[i] : __shfl_sync(0xffffffffu, scale[i], (lane & 28) + j / (GROUP / 32));
#pragma unroll
                            for (int b = 0; b < NT; ++b) {
                                acc[a][b][2 * h] = fmaf(f, sub[a][b][2 * h], acc[a][b][2 * h]);
                                acc[a][b][2 * h + 1] = fmaf(f, sub[a][b][2 * h + 1], acc[a][b][2 * h + 1]);
                            }
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(s));
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
        // The ring is read by every warp before partials lie over it.
        __syncthreads();
        if (*abort_flag) __syncthreads();
        float* mine = part + wk * Gm::MT * Gm::PITCH;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = 32 * wr + 16 * a + 8 * (e >> 1) + g, m = 8 * b + 2 * c + (e & 1);
                    mine[m * Gm::PITCH + n] = acc[a][b][e];
                }
    }
    if (warp == kWarps) {
        __syncthreads();
        if (*abort_flag) {
            // Copies that nobody waited for land before the ring is reused.
            if (lane == 0)
                for (int j = issued - S > 0 ? issued - S : 0; j < issued; ++j) {
                    const unsigned long long t0 = globaltimer_ns();
                    while (!mbar_try_wait(full_bar(j % S), static_cast<uint32_t>((j / S) & 1)))
                        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
                }
            __syncthreads();
        }
    }
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // CTA `rank` adds the cluster's partials of its share of the outputs, in
    // order, four adjacent ones a thread.
    const int rows = min(Gm::MT, p.M - m0);
    const int total = rows * (R / 4);
    const uint32_t part_addr = smem_addr(part);
    for (int i = total * rank / split + static_cast<int>(threadIdx.x); i < total * (rank + 1) / split; i += kThreads) {
        const int m = i / (R / 4), col = i % (R / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int r = 0; r < split; ++r)
#pragma unroll
            for (int k = 0; k < Gm::WK; ++k) {
                const int at = (k * Gm::MT + m) * Gm::PITCH + col;
                const float4 u = split == 1 ? *reinterpret_cast<const float4*>(part + at)
                                            : ld_cluster_f4(mapa_shared(part_addr + 4u * at, static_cast<uint32_t>(r)));
                v.x += u.x;
                v.y += u.y;
                v.z += u.z;
                v.w += u.w;
            }
        const int n = n0 + col;
        T* out = static_cast<T*>(p.C) + static_cast<long long>(m0 + m) * p.ldc + n;
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < p.N) out[e] = of_f32<T>(f[e]);
    }
    if (split > 1) cluster_sync_all();  // the peers have read this CTA's partials
}

// Eight weights (one 32-bit word) a thread, group/8 threads a group.
template <typename T, typename S>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4QuantLaunch p) {
    const long long words = p.K / 8;
    const long long t = blockIdx.x * 256ll + threadIdx.x;
    const bool in = t < p.N * words;
    // Threads past the end repeat the last word, so that whole warps shuffle.
    const long long u = in ? t : p.N * words - 1;
    const long long j = u / words, k = u % words * 8;
    const T* w = static_cast<const T*>(p.w) + j * p.ld + k;
    float v[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = f32_of(w[e]);
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
    for (int o = p.group / 16; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    S s16 = of_f32<S>(p.zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    if (f32_of(s16) < 1.17549435e-38f) s16 = of_f32<S>(0.0f);  // below 2^-126, 1/scale overflows
    const float s = f32_of(s16);
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    const float z = p.zeros ? fminf(rintf(-lo * inv), 15.0f) : 8.0f;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaxf(rintf(v[e] * inv) + z, 0.0f), 15.0f);
        word |= static_cast<uint32_t>(q) << (4 * e);
    }
    if (!in) return;
    uint8_t* out = p.W + j * p.ldw + k / 2;
    for (int e = 0; e < 4; ++e) out[e] = static_cast<uint8_t>(word >> (8 * e));
    if (k % p.group == 0) {
        static_cast<S*>(p.scales)[j * p.lds + k / p.group] = s16;
        if (p.zeros) p.zeros[j * p.ldz + k / p.group] = static_cast<uint8_t>(z);
    }
}

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

// The packed weights as N rows of K/2 bytes, boxes of R rows by one K block,
// swizzled over the block's bytes.
template <int NT>
bool encode_w(CUtensorMap* map, const W4Launch& L) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(L.K / 2), static_cast<cuuint64_t>(L.N)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(L.ldw)};
    cuuint32_t box[2] = {Geo<NT>::KS / 2, Geo<NT>::R};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(L.W), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              Geo<NT>::KS == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x as K/32 slices of M rows by 32 elements (64 bytes): a box lands slice by
// slice, so that a warp's 16-byte reads of eight rows touch every bank once.
template <int NT>
bool encode_x(CUtensorMap* map, const W4Launch& L, int x_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {32, static_cast<cuuint64_t>(L.M), static_cast<cuuint64_t>(L.K / 32)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(L.ldx * 2), 64};
    cuuint32_t box[3] = {32, static_cast<cuuint32_t>(x_rows), Geo<NT>::KS / 32};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, L.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(L.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int NT, int GROUP>
int launch_one(const W4Launch& L, cudaStream_t stream) {
    using Gm = Geo<NT>;
    W4Params p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.K = static_cast<int>(L.K);
    p.groups = static_cast<int>(L.K / GROUP);
    p.blocks = static_cast<int>((L.K + Gm::KS - 1) / Gm::KS);
    p.tiles_m = static_cast<int>((L.M + Gm::MT - 1) / Gm::MT);
    p.x_rows = static_cast<int>(L.M < Gm::MT ? L.M : Gm::MT);
    p.scales = L.scales;
    p.lds = L.lds;
    p.zeros = L.zeros;
    p.ldz = L.ldz;
    p.C = L.C;
    p.ldc = L.ldc;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * ((L.N + Gm::R - 1) / Gm::R);
    const int sms = tc_current_device_sms();
    if (sms <= 0) return GEMM_ERR_CUDA;
    // Two CTAs an SM.  Cut K over up to 8 CTAs while they are all resident and
    // each keeps two blocks.
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * sms && p.blocks / (2 * split) >= 2) split *= 2;
    p.split = split;
    if (tiles * split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    const int slot = Gm::W_BYTES + ((p.x_rows * Gm::KS * 2 + 127) & ~127);
    constexpr int kBudget = 110 * 1024;
    int stages = (kBudget - 1024) / slot;
    if (stages > kMaxStages) stages = kMaxStages;
    p.stages = stages;
    static_assert(Gm::PART_FLOATS * 4 <= 3 * Gm::W_BYTES && 3 * (Gm::W_BYTES + Gm::MT * Gm::KS * 2) <= kBudget - 1024,
                  "the partials lie over the ring, which has three stages at least");
    CUtensorMap tmW, tmX;
    if (!encode_w<NT>(&tmW, L) || !encode_x<NT>(&tmX, L, p.x_rows)) return GEMM_ERR_LAUNCH;
    auto kernel = w4_kernel<BF16, NT, GROUP>;
    {
        static std::mutex mu;
        static bool done[64] = {};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GEMM_ERR_CUDA;
        std::lock_guard<std::mutex> g(mu);
        if (!done[dev]) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBudget) != cudaSuccess)
                return GEMM_ERR_LAUNCH;
            done[dev] = true;
        }
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(1024 + stages * slot);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p) == cudaSuccess && cudaGetLastError() == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_LAUNCH;
}

template <int NT>
int launch_group(const W4Launch& L, cudaStream_t stream) {
    if (L.group == 32) return L.bf16 ? launch_one<true, NT, 32>(L, stream) : launch_one<false, NT, 32>(L, stream);
    if (L.group == 64) return L.bf16 ? launch_one<true, NT, 64>(L, stream) : launch_one<false, NT, 64>(L, stream);
    return L.bf16 ? launch_one<true, NT, 128>(L, stream) : launch_one<false, NT, 128>(L, stream);
}

template <typename T>
void quantize_of(const W4QuantLaunch& L, unsigned grid, cudaStream_t stream) {
    if (L.scale_bf16) w4_quantize_kernel<T, __nv_bfloat16><<<grid, 256, 0, stream>>>(L);
    else w4_quantize_kernel<T, __half><<<grid, 256, 0, stream>>>(L);
}

}  // namespace

int w4_launch(const W4Launch& L, cudaStream_t stream) {
    // One tile of up to 8, 16 or 32 rows of x; more rows are tiles of 32, each
    // of which reads the weights once more.
    if (L.M <= 8) return launch_group<1>(L, stream);
    if (L.M <= 16) return launch_group<2>(L, stream);
    return launch_group<4>(L, stream);
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
