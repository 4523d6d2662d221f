// What the head's tensor-core products share: the pipeline's sizes, 16-bit pairs, fp32
// values as three bf16 parts, copies of operands in the layout TMA reads, tensor
// maps and launches of CTA pairs.  Each translation unit has its own.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "head_device.cuh"
#include "head_internal.h"
#include "head_parts.cuh"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kBM = 128, kBK = 64;            // MMA rows; K elements per stage (128 bytes)
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxRing = 8;
// Epilogue warps.  PROMOTE: sixteen, so that a segment's sums are out of tensor
// memory well within the next segment's MMAs (eight took 2400 cycles for 2048).
__host__ __device__ constexpr int epi_warps(bool promote) { return promote ? 16 : 8; }
constexpr int kStageWarpBytes = 32 * 17 * 4;  // epilogue staging per warp: 32 rows of 17 words
constexpr int kSmemMost = 227 * 1024;

// The products of parts of two fp32 values that matter, the small ones first.
__device__ __constant__ int kPartA[6] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ int kPartB[6] = {0, 2, 1, 0, 1, 0};

// 32 consecutive values of a row as 16-bit pairs.
template <bool BF16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

template <bool BF16> __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    unpack2f(widen_pair<std::conditional_t<BF16, __nv_bfloat16, __half>>(w), a, b);
}

// Rows of T as [rows][parts * pitch] 16-bit values for the tensor cores, zero
// past `cols`, and zero for rows whose target does not count (target given):
// their weight in dw is zero, which would not hide a NaN.
template <typename T, int PARTS>
__device__ __forceinline__ void pack_parts(const T* src, int64_t stride, int64_t rows, int cols, int pitch, int vec,
                                           const int64_t* target, int vocab, int64_t ignore, uint16_t* dst,
                                           int64_t block, int64_t blocks) {
    const int per = pitch / 8;
    const int64_t total = rows * per;
    for (int64_t i = block * blockDim.x + threadIdx.x; i < total; i += blocks * blockDim.x) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        bool keep = true;
        if (target) {
            const int64_t t = target[row];
            keep = t != ignore && t >= 0 && t < vocab;
        }
        const T* s = src + row * stride + c;
        uint16_t* d = dst + row * (int64_t)PARTS * pitch + c;
        if constexpr (PARTS == 1) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (keep) {
                if (vec && c + 8 <= cols) {
                    v = *reinterpret_cast<const uint4*>(s);
                } else {
                    uint16_t e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = c + j < cols ? reinterpret_cast<const uint16_t*>(s)[j] : 0;
                    v = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                   e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                }
            }
            *reinterpret_cast<uint4*>(d) = v;
        } else {
            float x[8], q[8][3];
            if (vec && keep && c + 8 <= cols) {
                const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
                x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
                x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = keep && c + j < cols ? to_f32(s[j]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(x[j], q[j]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4*>(d + (int64_t)k * pitch) =
                    make_uint4(pack2<true>(q[0][k], q[1][k]), pack2<true>(q[2][k], q[3][k]),
                               pack2<true>(q[4][k], q[5][k]), pack2<true>(q[6][k], q[7][k]));
        }
    }
}

// ------------------------------------------------------------------ host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef CUresult (*PFN_encode_t)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A row-major 16-bit matrix read in boxes of 64 columns (128 bytes, swizzled)
// by `box_rows` rows; zeros outside.
bool make_map(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    static PFN_encode_t enc = reinterpret_cast<PFN_encode_t>(driver_entry("cuTensorMapEncodeTiled"));
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t str[1] = {(cuuint64_t)pitch * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
               const_cast<void*>(base), dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool allow_smem(const void* kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) == cudaSuccess;
}

constexpr int kFixedSmem = 1024 + (2 * kMaxRing + 5) * 8 + 24;

cudaError_t launch_clusters(const void* kern, int grid, int threads, int ctas, int smem, cudaStream_t st, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

void take(size_t& at, size_t& off, size_t bytes) {
    off = at;
    at += align_up(bytes, 1024);
}

// A matrix as the tensor cores read it: base, columns and row pitch.
struct Operand { const void* base; int64_t cols, pitch; };

uint8_t* aligned_base(void* ws) {
    return reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(ws), 1024));
}

}  // namespace

}  // namespace conv2d_gb300
