// Dropout from a counter-based generator: y = residual + keep x / (1 - p).
//
// One Philox4x32-10 call (Salmon et al., "Parallel random numbers: as easy as
// 1, 2, 3", 2011) yields eight 16-bit words, one for each of eight adjacent
// elements: the high half of the 32-bit number that is compared with
// round(p 2^32).  The low half decides only where the high half equals the
// threshold's (one element in 65536), so the second call that yields the low
// halves runs only for those blocks: the comparison is the exact 32-bit one at
// half the multiplications, which would otherwise bound the 16-bit types.
// A thread owns blocks of eight elements; the mask exists in registers only.
//
// Memory bounds it: 16384 x 2048 bf16 with a residual 31.4 us (6.4 TB/s), fp32
// 8192 x 4096 with one 58.1 us (6.9 TB/s); without a residual the generator's
// share shows (26.3 us, 5.1 TB/s).  Seven rows of 1001 take 1.8 us.
#include <math.h>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

struct DropParams {
    int64_t rows, cols, xs, rs, ys;
    int64_t blocks;              // blocks of eight elements of the whole tensor
    uint32_t k0, k1, off0, off1;
    uint32_t threshold;          // dropped below it
    int all;                     // threshold 2^32: nothing is kept
    float scale;
    const void *x, *r;
    void* y;
};

// The 32-bit numbers of block b's eight elements.  Their high halves come from
// one Philox call; what stands below a high half is meaningless unless it ties
// with the threshold's, and then the second call fills the low halves in.
__device__ __forceinline__ void numbers(const DropParams& p, int64_t b, uint32_t (&n)[8]) {
    if (p.all) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = 0u;         // below the threshold, 2^32 - 1 here
        return;
    }
    uint32_t c[4] = {(uint32_t)b, (uint32_t)((uint64_t)b >> 32), p.off0, p.off1};
    philox(c, p.k0, p.k1);
    const uint32_t base = p.threshold & 0xffff0000u;
    uint32_t nearest = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        n[i] = i & 1 ? c[i >> 1] : c[i >> 1] << 16;
        nearest = min(nearest, n[i] - base);           // below 2^16: the high halves are equal
    }
    if (nearest < 0x10000u) {
        uint32_t l[4] = {(uint32_t)b, (uint32_t)((uint64_t)b >> 32), p.off0, p.off1 | 0x80000000u};
        philox(l, p.k0, p.k1);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = (n[i] & 0xffff0000u) | (i & 1 ? l[i >> 1] >> 16 : l[i >> 1] & 0xffffu);
    }
}

// How a call's blocks of eight lie: FLAT, adjacent in every tensor; ROWS,
// inside rows a multiple of eight long; both 16-byte aligned.  SINGLE: each
// element finds its own row and column.
enum Lie { FLAT = 0, ROWS = 1, SINGLE = 2 };

// One block a thread; six blocks of threads an SM (40 registers) cover the
// loads of some with the generator's arithmetic of others.
template <typename T, int LIE, bool RESIDUAL>
__global__ void __launch_bounds__(256, 6) dropout_kernel(const DropParams p) {
    constexpr int V = 16 / (int)sizeof(T), L = 8 / V;  // a block is one load of 16-bit values, two of fp32
    pdl_wait();
    const T* x = static_cast<const T*>(p.x);
    const T* r = static_cast<const T*>(p.r);
    T* y = static_cast<T*>(p.y);
    const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (b >= p.blocks) return;
    const int64_t total = p.rows * p.cols;
    int64_t e0 = b * 8, row = 0, col = e0;
    if constexpr (LIE != FLAT) {
        row = e0 / p.cols;
        col = e0 - row * p.cols;
    }
    if (LIE != SINGLE && e0 + 8 <= total) {
        Vec<T, V> vx[L], vr[L];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            vx[l] = *reinterpret_cast<const Vec<T, V>*>(x + row * p.xs + col + l * V);
            if (RESIDUAL) vr[l] = *reinterpret_cast<const Vec<T, V>*>(r + row * p.rs + col + l * V);
        }
        uint32_t n[8];
        numbers(p, b, n);
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float f[V], g[V];
            widen(vx[l], f);
            if (RESIDUAL) widen(vr[l], g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[i] = n[l * V + i] >= p.threshold ? f[i] * p.scale : 0.f;
                if (RESIDUAL) f[i] += g[i];
            }
            *reinterpret_cast<Vec<T, V>*>(y + row * p.ys + col + l * V) = narrow<T, V>(f);
        }
    } else {
        uint32_t n[8];
        numbers(p, b, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (e0 + i < total) {
                float f = n[i] >= p.threshold ? to_f32(x[row * p.xs + col]) * p.scale : 0.f;
                if (RESIDUAL) f += to_f32(r[row * p.rs + col]);
                y[row * p.ys + col] = from_f32<T>(f);
                if (LIE == FLAT) {
                    ++col;
                } else if (++col == p.cols) {
                    col = 0;
                    ++row;
                }
            }
        }
    }
}

template <typename T> cudaError_t run(const DropParams& p, int lie, cudaStream_t st) {
    const int64_t grid = (p.blocks + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;      // 2^42 elements
#define DROP(LIE) (p.r ? dropout_kernel<T, LIE, true> : dropout_kernel<T, LIE, false>)
    auto kern = lie == FLAT ? DROP(FLAT) : lie == ROWS ? DROP(ROWS) : DROP(SINGLE);
#undef DROP
    return launch_after(kern, dim3((unsigned)grid), dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_dropout(const dropout_desc& d, const void* x, int64_t xs, const void* residual, int64_t rs, void* y,
                           int64_t ys, uint64_t seed, uint64_t offset, cudaStream_t st) {
    DropParams p{};
    p.rows = d.rows; p.cols = d.cols; p.xs = xs; p.rs = rs; p.ys = ys;
    const bool flat = xs == d.cols && ys == d.cols && (!residual || rs == d.cols);
    if (flat) {
        p.rows = 1;
        p.cols = p.xs = p.rs = p.ys = d.rows * d.cols;
    }
    p.blocks = (d.rows * d.cols + 7) / 8;
    p.k0 = (uint32_t)seed; p.k1 = (uint32_t)(seed >> 32);
    p.off0 = (uint32_t)offset; p.off1 = (uint32_t)(offset >> 32);
    const uint64_t threshold = (uint64_t)nearbyint(d.p * 4294967296.0);
    p.all = threshold >> 32 != 0;
    p.threshold = p.all ? 0xffffffffu : (uint32_t)threshold;
    p.scale = d.p < 1.0 ? (float)(1.0 / (1.0 - d.p)) : 0.f;
    p.x = x; p.r = residual; p.y = y;
    const int64_t e = (int64_t)elem_bytes(d.dtype);
    const bool aligned = aligned_to(x, 16) && aligned_to(y, 16) && aligned_to(residual, 16);
    const bool rows = d.cols % 8 == 0 && xs * e % 16 == 0 && ys * e % 16 == 0 && (!residual || rs * e % 16 == 0);
    const int lie = !aligned ? SINGLE : flat ? FLAT : rows ? ROWS : SINGLE;
    switch (d.dtype) {
        case CONV2D_F32: return run<float>(p, lie, st);
        case CONV2D_F16: return run<__half>(p, lie, st);
        default: return run<__nv_bfloat16>(p, lie, st);
    }
}

}  // namespace conv2d_gb300
