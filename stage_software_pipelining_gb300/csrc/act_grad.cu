// act_grad.cu -- dz = dy act'(z) and the bias gradient, the sum of dz's rows.
//
// One pass over dy and z, bound by memory.  A CTA, or a cluster of them that
// shares the rows, owns a strip of columns: every thread adds its rows' unrounded
// values in fp32, a CTA its threads', and the first CTA of the cluster the others'
// through distributed shared memory, all in a fixed order and without a workspace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "activation.cuh"
#include "internal.h"
#include "linear.h"
#include "product.cuh"
#include "ptx.cuh"

namespace ssp {
namespace {

constexpr int kMostParts = 16;  // CTAs of a cluster

struct Params {
    int M, N;
    int rows;  // of a CTA
    int act;
    const uint16_t* dy;
    long long lddy;
    const uint16_t* pre;
    long long ldp;
    uint16_t* dz;
    long long lddz;
    float* dbias;
    const float* addend;
};

template <int VEC>
struct Values {
    uint32_t u[VEC / 2];
};
template <>
struct Values<1> {
    uint32_t u[1];
};

// VEC adjacent values, of which `left` are in the row (one: and a zero beside it).
template <int VEC>
__device__ __forceinline__ Values<VEC> load(const uint16_t* p, int left) {
    Values<VEC> v;
    if constexpr (VEC == 1) {
        v.u[0] = *p;
    } else if (left >= VEC) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v.u[0] = q.x;
        v.u[1] = q.y;
        v.u[2] = q.z;
        v.u[3] = q.w;
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            v.u[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
    }
    return v;
}

// Strips of VEC * GROUPS columns; ROWS rows at a time.  VEC = 8 wants rows on
// 16-byte boundaries.
template <bool BF16, int VEC, int ACT, int GROUPS, int THREADS>
__device__ __forceinline__ void pass(const Params& p, int r0, int r1, int c, Pair (&sum)[(VEC + 1) / 2]) {
    constexpr int ROWS = THREADS / GROUPS;
    constexpr int AHEAD = 4;  // rows of a thread whose loads are under way together
    const int left = p.N - c;
    if (left <= 0) return;
    for (int r = r0 + static_cast<int>(threadIdx.x) / GROUPS; r < r1; r += AHEAD * ROWS) {
        Values<VEC> dy[AHEAD], z[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const long long row = r + a * ROWS;
            if (row < r1) {
                dy[a] = load<VEC>(p.dy + row * p.lddy + c, left);
                if (ACT != LINEAR_ACT_NONE) z[a] = load<VEC>(p.pre + row * p.ldp + c, left);
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const long long row = r + a * ROWS;
            if (row >= r1) break;
            uint32_t out[VEC == 8 ? 4 : 1];
#pragma unroll
            for (int i = 0; i < (VEC + 1) / 2; ++i) {
                Pair g = unpack16_pair<BF16>(dy[a].u[i]);
                if constexpr (ACT != LINEAR_ACT_NONE) g = mul2(g, derivative<ACT>(unpack16_pair<BF16>(z[a].u[i])));
                sum[i] = add2(sum[i], g);
                out[i] = pack16<BF16>(g);
            }
            if (p.dz) {
                uint16_t* d = p.dz + row * p.lddz + c;
                if constexpr (VEC == 1) {
                    *d = static_cast<uint16_t>(out[0]);
                } else if (left >= VEC) {
                    *reinterpret_cast<uint4*>(d) = make_uint4(out[0], out[1], out[2], out[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (i < left) d[i] = static_cast<uint16_t>(out[i / 2] >> (16 * (i & 1)));
                }
            }
        }
    }
}

template <bool BF16, int VEC, int GROUPS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) act_grad_kernel(const Params p) {
    constexpr int COLS = GROUPS * VEC, WARPS = THREADS / 32;
    __shared__ float sums[WARPS][COLS];
    __shared__ float total[COLS];
    griddep_wait();
    griddep_launch_dependents();
    const int rank = static_cast<int>(blockIdx.y), parts = static_cast<int>(gridDim.y);  // a cluster is a column of the grid
    const int col0 = static_cast<int>(blockIdx.x) * COLS;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int c = col0 + static_cast<int>(threadIdx.x % GROUPS) * VEC;
    const int r0 = static_cast<int>(min(static_cast<long long>(p.M), static_cast<long long>(rank) * p.rows));
    const int r1 = static_cast<int>(min(static_cast<long long>(p.M), static_cast<long long>(r0) + p.rows));
    Pair sum[(VEC + 1) / 2] = {};
    if (p.act == LINEAR_ACT_NONE)
        pass<BF16, VEC, LINEAR_ACT_NONE, GROUPS, THREADS>(p, r0, r1, c, sum);
    else
        with_activation(p.act, [&](auto a) { pass<BF16, VEC, decltype(a)::value, GROUPS, THREADS>(p, r0, r1, c, sum); });
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
        float2 s = both(sum[i]);
#pragma unroll
        for (int d = GROUPS; d < 32; d *= 2) {  // lanes that hold the same columns
            s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
        }
        if (lane < GROUPS) {
            sums[threadIdx.x / 32][lane * VEC + 2 * i] = s.x;
            if (VEC > 1) sums[threadIdx.x / 32][(lane * VEC + 2 * i + 1) % COLS] = s.y;
        }
    }
    __syncthreads();
    if (threadIdx.x < COLS) {
        float s = 0.0f;
#pragma unroll 8
        for (int w = 0; w < WARPS; ++w) s += sums[w][threadIdx.x];
        total[threadIdx.x] = s;
    }
    if (parts > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0 && threadIdx.x < COLS && col0 + static_cast<int>(threadIdx.x) < p.N) {
        const int j = col0 + static_cast<int>(threadIdx.x);
        float s = total[threadIdx.x];
#pragma unroll 1
        for (int r0 = 1; r0 < parts; r0 += 8) {  // eight on their way together
            float other[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                other[r] = ld_cluster_f32(mapa_shared(smem_addr(&total[threadIdx.x]), static_cast<uint32_t>(min(r0 + r, parts - 1))));
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r0 + r < parts) s += other[r];
        }
        p.dbias[j] = p.addend ? p.addend[j] + s : s;
    }
    if (parts > 1) cluster_sync_all();  // the others' sums have been read
}

// CTAs that share a strip's rows: as many as have a few each and run at once
// (fewer CTAs in a second round than in the first leave memory idle).  A sum's are
// a cluster, of `widest` at most.
int parts_of(const ActGradLaunch& L, int cols, int groups, int threads, int widest = 8) {
    const int64_t strips = (L.N + cols - 1) / cols;
    const int64_t slots = static_cast<int64_t>(tc_current_device_sms()) * (1024 / threads);
    const int64_t rows = 4 * (threads / groups);
    int64_t parts = (L.M + rows - 1) / rows;
    int64_t most = slots / strips;
    if (L.dbias && most > widest) most = widest;
    if (most < 1) most = 1;
    if (parts > most) parts = most;
    return static_cast<int>(parts < 1 ? 1 : parts);
}

// Clusters of more than eight CTAs are allowed once a device.
bool allow_wide(const void* kernel, bool (&done)[64]) {
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> g(mu);
    if (!done[dev])
        done[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    return done[dev];
}

template <bool BF16, int VEC, int GROUPS, int THREADS>
int launch(const ActGradLaunch& L, cudaStream_t stream) {
    constexpr int COLS = VEC * GROUPS;
    // Sixteen CTAs a cluster, two an SM, where all strips' clusters run at once: as
    // many as clusters of eight, one an SM (28491 x 210, gelu: 21.4 us, of eight CTAs 34.5).
    int widest = 8;
    if constexpr (COLS == 32) {
        static bool done[64] = {};
        int resident[9];
        if (L.dbias && product_resident_ctas(resident) && (L.N + COLS - 1) / COLS <= resident[8] / 8 &&
            allow_wide(reinterpret_cast<const void*>(act_grad_kernel<BF16, VEC, GROUPS, THREADS>), done))
            widest = kMostParts;
    }
    const int parts = parts_of(L, COLS, GROUPS, THREADS, widest);
    Params p = {};
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.act = L.act;
    p.dy = static_cast<const uint16_t*>(L.dy);
    p.lddy = L.lddy;
    p.pre = static_cast<const uint16_t*>(L.pre);
    p.ldp = L.ldp;
    p.dz = static_cast<uint16_t*>(L.dz);
    p.lddz = L.lddz;
    p.dbias = L.dbias;
    p.addend = L.addend;
    p.rows = static_cast<int>((L.M + parts - 1) / parts);
    const int64_t strips = (L.N + COLS - 1) / COLS;
    ProductConfig c(strips, parts, THREADS, 0, stream);
    c.cfg.gridDim = dim3(static_cast<unsigned>(strips), static_cast<unsigned>(parts));
    c.attr[1].val.clusterDim.x = 1;
    c.attr[1].val.clusterDim.y = static_cast<unsigned>(parts);
    if (!L.dbias) c.cfg.numAttrs = 1;  // no cluster
    return product_finish(cudaLaunchKernelEx(&c.cfg, act_grad_kernel<BF16, VEC, GROUPS, THREADS>, p));
}

// Strips of 64 columns, 128 bytes a row, and CTAs of 512 threads, two an SM.  Where
// clusters of eight of them leave many places empty (a sum over many rows of few
// columns), strips of 32 columns: 32768 x 1024 in strips of 64 takes 69 us, of 32
// 39.  Where rows are many and the strips fill one CTA an SM better than two, CTAs of
// 1024 threads.
template <bool BF16>
int launch_vectors(const ActGradLaunch& L, cudaStream_t stream) {
    const int64_t sms = tc_current_device_sms();
    if (L.dbias && L.M >= 1024 && (L.N + 63) / 64 * 8 <= sms) return launch<BF16, 8, 4, 512>(L, stream);
    if (L.M >= 4096 && 2 * parts_of(L, 64, 8, 1024) > parts_of(L, 64, 8, 512)) return launch<BF16, 8, 8, 1024>(L, stream);
    return launch<BF16, 8, 8, 512>(L, stream);
}

}  // namespace

int act_grad_launch(const ActGradLaunch& L, cudaStream_t stream) {
    auto fits = [&](const void* p, int64_t ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld % 8 == 0 || L.M <= 1));
    };
    const bool vec = fits(L.dy, L.lddy) && fits(L.pre, L.ldp) && fits(L.dz, L.lddz);
    if (L.bf16) return vec ? launch_vectors<true>(L, stream) : launch<true, 1, 32, 512>(L, stream);
    return vec ? launch_vectors<false>(L, stream) : launch<false, 1, 32, 512>(L, stream);
}

}  // namespace ssp
