// product.cuh -- what the two kernels of the training operators' products share:
// the operands' layouts in shared memory, their tensor maps, the waits, and the
// conversions of an epilogue.
//
// Operands are 16-bit and come in either order of the matrix in memory.  A stage
// of the ring holds K = 64 of both:
//   * K-major (adjacent k): rows of 64 k, one 128-byte swizzle row each;
//   * MN-major (adjacent rows or columns of the result, as dz and x lie for
//     dz^T x): chunks of 64 of them, a 128-byte swizzle row a k, 8 KB a chunk.
// Either way 128 rows or columns of a stage are 16 KB.  All chunks of an MN-major
// stage come by one copy, through a map that has the chunk as a dimension of its
// own, 64 elements from one to the next; a copy a chunk cost 7 % of the pair
// kernel's time for each such operand (4096^3: 82 us, with chunks by themselves 89
// for one and 98 for two).  Where a tile's chunks reach past the matrix they come
// one by one, from a map that ends where the matrix does.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "internal.h"
#include "linear.h"
#include "ptx.cuh"
#include "tensor_copy.cuh"

namespace ssp {

constexpr int PK = 64;                    // K of a stage
constexpr int PUMMA_K = 16;               // K per tcgen05.mma (kind::f16)
constexpr int P_TILE_BYTES = 128 * PK * 2;  // 128 rows or columns of a stage: 16 KB
constexpr int P_CHUNK_BYTES = 64 * PK * 2;  // an MN-major chunk of a stage: 8 KB
constexpr int kProductSmem = 227 * 1024;
constexpr int P_PRODUCER = 0, P_MMA = 1, P_EPILOGUE = 2;

// Shared-memory matrix descriptor of an operand: 8-row groups 1024 bytes apart,
// 128-byte swizzle; the leading offset is that of MN-major chunks.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int mn) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
           (static_cast<uint64_t>(mn ? P_CHUNK_BYTES / 16 : 1) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// The step of a K = 16 product in a descriptor's address (16-byte units): 32
// bytes along the rows, or 16 rows.
__device__ __forceinline__ uint32_t operand_step(int mn) { return mn ? 2048u / 16u : 32u / 16u; }

// Instruction descriptor (kind::f16): D fp32 (bit 4), types at bits 7 and 10 (0
// fp16, 1 bf16), MN-major operands at bits 15 and 16, N >> 3 at bits 17..22, M >>
// 4 at bits 24..28.
inline uint32_t product_instruction(int m, int n, int bf16, int a_mn, int b_mn) {
    const uint32_t t = bf16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void record_product_timeout(GemmDeviceStatus* status, int role, int iter) {
    if (atomicCAS(&status->code, 0, GEMM_ERR_TIMEOUT) == 0) {
        status->block = blockIdx.x;
        status->role = role;
        status->iter = iter;
        __threadfence();
    }
}

// Wait for the phase of `bar` with parity `parity`; false after limit_ns or
// once another role has raised the abort flag.  PAIR: the peer CTA's flag is
// raised too.
template <bool PAIR>
__device__ __forceinline__ bool product_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                             unsigned long long limit_ns, GemmDeviceStatus* status, int role, int iter) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                record_product_timeout(status, role, iter);
                *abort = 1;
                if constexpr (PAIR)
                    st_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(abort)), (cluster_ctarank() & 1u) ^ 1u), 1u);
                return false;
            }
        }
    }
}

// Two fp32 values in 16 bits, and back.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
    if constexpr (BF16) {
        const __nv_bfloat162 o = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&o);
    } else {
        const __half2 o = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&o);
    }
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(Pair p) {
    const float2 v = both(p);
    return pack16<BF16>(v.x, v.y);
}
__device__ __forceinline__ uint32_t pack16(bool bf16, float x, float y) {
    return bf16 ? pack16<true>(x, y) : pack16<false>(x, y);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
}
__device__ __forceinline__ float2 unpack16(bool bf16, uint32_t v) {
    return bf16 ? unpack16<true>(v) : unpack16<false>(v);
}
template <bool BF16>
__device__ __forceinline__ Pair unpack16_pair(uint32_t v) {
    const float2 f = unpack16<BF16>(v);
    return make_pair2(f.x, f.y);
}
template <bool BF16>
__device__ __forceinline__ float load16(const void* p, long long i) {
    if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ float load16(bool bf16, const void* p, long long i) {
    return bf16 ? load16<true>(p, i) : load16<false>(p, i);
}

// t^n for n = 0, 1, 2.  (t comes from the kernel before this one, which may still
// run when this one starts: no load here goes through the read-only path.)
__device__ __forceinline__ float power_of(const float* t, int b, int n) {
    const float v = n ? t[b] : 1.0f;
    return n == 2 ? v * v : v;
}

// ---------------------------------------------------------------- host side
// Row-major matrices of `cols` elements a row in boxes of box_cols x box_rows.
inline bool encode_matrices(CUtensorMap* map, CUtensorMapDataType type, int size, CUtensorMapSwizzle swizzle,
                            const ProductMatrix& m, int64_t rows, int64_t cols, int64_t batch, int box_cols,
                            int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int64_t unit = 16 / size;
    // A single row's leading dimension, or a single matrix's stride, is not used
    // but has to fit.
    const int64_t ld = rows > 1 ? m.ld : (cols + unit - 1) / unit * unit;
    const int64_t stride = batch > 1 ? m.stride : ld;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * size), static_cast<cuuint64_t>(stride * size)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, type, 3, const_cast<void*>(m.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline CUtensorMapDataType type16(int bf16) {
    return bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// An operand with `len` rows or columns of the result and sums of K, `tile` of them
// a stage.  `map`: boxes of 64 k by `tile`, or (MN-major) all chunks of a stage at
// once, for tiles that lie within the matrix; `edge`: (MN-major) boxes of 64 rows or
// columns by 64 k.
inline bool encode_operand(CUtensorMap* map, CUtensorMap* edge, const ProductMatrix& m, int mn, int bf16, int64_t len,
                           int64_t K, int64_t batch, int tile) {
    if (!mn) {
        *edge = {};
        return encode_matrices(map, type16(bf16), 2, CU_TENSOR_MAP_SWIZZLE_128B, m, len, K, batch, PK, tile);
    }
    if (!encode_matrices(edge, type16(bf16), 2, CU_TENSOR_MAP_SWIZZLE_128B, m, K, len, batch, 64, PK)) return false;
    const int chunks = (tile + 63) / 64;
    if (len < 64 * chunks) {  // no tile lies within the matrix
        *map = *edge;
        return true;
    }
    auto fn = tensor_map_encoder();
    const int64_t ld = K > 1 ? m.ld : (len + 7) / 8 * 8;
    const int64_t stride = batch > 1 ? m.stride : ld;
    // Elements of a chunk start where the last one's still end within the row.
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(len - 64 * (chunks - 1)), static_cast<cuuint64_t>(K),
                          static_cast<cuuint64_t>(chunks), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld * 2), 128, static_cast<cuuint64_t>(stride * 2)};
    cuuint32_t box[4] = {64, PK, static_cast<cuuint32_t>(chunks), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, type16(bf16), 4, const_cast<void*>(m.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches overlap (programmatic serialization): a kernel's start runs beside the end
// of the one before it.  No kernel lets the next one start before griddep_wait: the
// one after next would take places on SMs before the next has its own (four 256 x
// 1024 orthogonalised, in a graph: 91 us, 106 with the two the other way round).
struct ProductConfig {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ProductConfig(int64_t grid, int cluster, int threads, size_t smem, cudaStream_t stream) {
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

// A launch's own status, after clearing whatever it left.
inline int product_finish(cudaError_t e) {
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace ssp
