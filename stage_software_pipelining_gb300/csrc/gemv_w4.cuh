// gemv_w4.cuh -- what the two kernels of the 4-bit product share: the unpacking
// of nibbles, bounded waits and the choice of the K split.
#pragma once
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
namespace w4 {

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

constexpr int KS = 256;        // K of a stage: one 128-byte swizzle row of nibbles
constexpr int kMaxStages = 8;

// Written by a wait that ran out; one a source file.
static __device__ GemmDeviceStatus g_status;

struct Params {
    int M, N, K;
    int tiles_m, groups;  // groups of a row
    int blocks;           // stages of K
    int split;            // CTAs of a cluster, each with a part of the stages
    int stages, x_rows;   // ring depth; rows of x in a stage
    uint32_t idesc;
    int s_vec, z_vec;     // rows of scales on 16-byte, of zeros on 8-byte boundaries
    const void* scales;
    long long lds;
    const uint8_t* zeros;
    long long ldz;
    void* C;
    long long ldc;
    unsigned long long wait_limit_ns;
    int withhold;         // block 0 leaves out this stage's copies (test hook), -1: none
};

// Wait for the phase of `bar` with parity `parity`; false after limit_ns or
// once another warp has raised the abort flag.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort,
                                         unsigned long long limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                if (atomicCAS(&g_status.code, 0, GEMM_ERR_TIMEOUT) == 0) {
                    g_status.block = blockIdx.x;
                    g_status.role = static_cast<int>(threadIdx.x >> 5);  // the warp
                    __threadfence();
                }
                *abort = 1;
                return false;
            }
        }
    }
}

// The same for a whole warp: true if the phase completed for every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          unsigned long long limit_ns) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort, limit_ns)) != 0;
}

// A warp's wait in two halves: a look at the barrier, whose latency (some 150
// clocks) passes under what stands between, and the wait for those that it
// found incomplete.
struct Wait {
    uint32_t bar, parity;
    bool ready;
    __device__ __forceinline__ Wait(uint32_t b, uint32_t ph) : bar(b), parity(ph), ready(mbar_test_wait(b, ph)) {}
    __device__ __forceinline__ bool done(volatile int* abort, unsigned long long limit_ns) const {
        return __all_sync(0xffffffffu, ready) || warp_wait(bar, parity, abort, limit_ns);
    }
};

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

// The zero point as unpack wants it: (128 + z) or (1024 + z) twice, and from
// that, for fp16, -(64 + z) twice (at 2^6 fp16 has 16 steps a unit).
template <bool BF16>
__device__ __forceinline__ uint32_t zero_of(uint32_t z) {
    return z * 0x00010001u + (BF16 ? 0x43004300u : 0x64006400u);
}
template <bool BF16>
__device__ __forceinline__ uint32_t zero16_of(uint32_t zero) {
    return BF16 ? 0u : (zero - 0x64006400u) * 16u + 0xd400d400u;
}

// x += scale * a and y += scale * b in one instruction, rounded as fmaf.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float scale) {
    uint64_t v, s, c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(s) : "f"(scale));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(x), "f"(y));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(v), "l"(s));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(c));
}

__device__ __forceinline__ void add4(float4& v, float4 u) {
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
}

// Four adjacent outputs of a row, those below N.
template <typename T>
__device__ __forceinline__ void store4(const Params& p, int m, int n, float4 v) {
    T* out = static_cast<T*>(p.C) + static_cast<long long>(m) * p.ldc + n;
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < p.N) out[e] = of_f32<T>(f[e]);
}

// ---------------------------------------------------------------- host side
// CTAs of a kernel that the current device holds at once, by cluster size
// 1..8; asked for once a device, with the kernel's shared-memory limit.
struct Residency {
    std::mutex mu;
    bool known[64] = {};
    int ctas[64][9] = {};

    bool get(const void* kernel, int threads, int smem, int (&out)[9]) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
        std::lock_guard<std::mutex> g(mu);
        if (!known[dev]) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return false;
            for (int c = 1; c <= 8; ++c) {
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = static_cast<unsigned>(c);
                attr.val.clusterDim.y = 1;
                attr.val.clusterDim.z = 1;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(static_cast<unsigned>(c));
                cfg.blockDim = dim3(static_cast<unsigned>(threads));
                cfg.dynamicSmemBytes = static_cast<size_t>(smem);
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                    cudaGetLastError();
                    n = 0;
                }
                ctas[dev][c] = n * c;
            }
            if (ctas[dev][1] <= 0) return false;
            known[dev] = true;
        }
        for (int c = 0; c <= 8; ++c) out[c] = ctas[dev][c];
        return true;
    }
};

// Cut K over 1 to 8 CTAs, a cluster, `least_blocks` stages each at least: the
// cut with the least time, counted in stages.  CTAs share the SMs evenly, so
// rounds of resident CTAs count in fractions, but a CTA's start and end (the
// cluster's barriers among them) cost about as much as eight stages each round
// (measured with every cut on 4096^2 to 28672 x 8192).
inline int choose_split(int64_t tiles, int blocks, int least_blocks, const int (&resident)[9]) {
    int split = 1;
    double least = 0.0;
    for (int c = 1; c <= 8 && (c == 1 || blocks / c >= least_blocks); ++c) {
        if (resident[c] <= 0) continue;
        const double rounds = static_cast<double>(tiles) * c / resident[c];
        const double whole = static_cast<double>((tiles * c + resident[c] - 1) / resident[c]);
        const double work = (rounds < 1.0 ? 1.0 : rounds) * ((blocks + c - 1) / c) + 8.0 * whole;
        if (c == 1 || work < 0.95 * least) {
            split = c;
            least = work;
        }
    }
    return split;
}

// Parameters that do not depend on the kernel's geometry.
inline Params params_of(const W4Launch& L) {
    Params p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.K = static_cast<int>(L.K);
    p.groups = static_cast<int>(L.K / L.group);
    p.blocks = static_cast<int>((L.K + KS - 1) / KS);
    p.scales = L.scales;
    p.lds = L.lds;
    p.zeros = L.zeros;
    p.ldz = L.ldz;
    p.s_vec = reinterpret_cast<uintptr_t>(L.scales) % 16 == 0 && (L.N == 1 || L.lds % 8 == 0);
    p.z_vec = reinterpret_cast<uintptr_t>(L.zeros) % 8 == 0 && (L.N == 1 || L.ldz % 8 == 0);
    p.C = L.C;
    p.ldc = L.ldc;
    const DebugHooks d = debug_hooks();
    p.wait_limit_ns = static_cast<unsigned long long>(d.wait_limit_ns);
    p.withhold = d.withhold_arrive;
    return p;
}

// Fill a plan query's answer in place of a launch.
inline int planned(const W4Launch& L, int kernel, int tile_rows, const Params& p, int64_t tiles, int smem) {
    if (tiles * p.split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    *L.plan = {kernel, tile_rows, p.split, p.stages, static_cast<int>(tiles * p.split), smem};
    return GEMM_OK;
}

// Launch with clusters of p.split CTAs, overlapping the previous kernel's end.
template <typename Kernel>
int launch(Kernel kernel, const CUtensorMap& tmW, const CUtensorMap& tmX, const Params& p, int64_t tiles, int threads,
           int smem, cudaStream_t stream) {
    if (tiles * p.split > 0x7fffffff) return GEMM_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p) == cudaSuccess && cudaGetLastError() == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_LAUNCH;
}

// The file's status word, read and reset (synchronous).
inline int read_and_clear_status(GemmDeviceStatus* out) {
    const GemmDeviceStatus zero = {0, 0, 0, 0};
    if (cudaMemcpyFromSymbol(out, g_status, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_status, &zero, sizeof(GemmDeviceStatus)) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
}

}  // namespace w4

// More than 16 rows of x (gemv_w4_tc.cu).
int w4_launch_tc(const W4Launch& L, cudaStream_t stream);
int w4_tc_read_and_clear_status(GemmDeviceStatus* out);

}  // namespace ssp
