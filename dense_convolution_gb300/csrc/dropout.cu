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
    uint32_t hi, lo;             // halves of the threshold
    int all, none;               // threshold 2^32 and 0
    float scale;
    const void *x, *r;
    void* y;
};

// Philox4x32-10: ten rounds of two 32x32-bit products.
__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
        const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ k0, n2 = (uint32_t)(a >> 32) ^ c[3] ^ k1;
        c[0] = n0; c[1] = (uint32_t)b; c[2] = n2; c[3] = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Bit i: element i of block b is kept.
__device__ __forceinline__ uint32_t keep_bits(const DropParams& p, int64_t b) {
    if (p.none) return 0xffu;
    if (p.all) return 0u;
    uint32_t c[4] = {(uint32_t)b, (uint32_t)((uint64_t)b >> 32), p.off0, p.off1};
    philox(c, p.k0, p.k1);
    uint32_t keep = 0, tie = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = i & 1 ? c[i >> 1] >> 16 : c[i >> 1] & 0xffffu;
        keep |= h > p.hi ? 1u << i : 0u;
        tie |= h == p.hi ? 1u << i : 0u;
    }
    if (tie) {
        uint32_t l[4] = {(uint32_t)b, (uint32_t)((uint64_t)b >> 32), p.off0, p.off1 | 0x80000000u};
        philox(l, p.k0, p.k1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = i & 1 ? l[i >> 1] >> 16 : l[i >> 1] & 0xffffu;
            if ((tie >> i & 1) && w >= p.lo) keep |= 1u << i;
        }
    }
    return keep;
}

// VECTOR: blocks of eight are whole, adjacent and 16-byte aligned in every
// tensor (rows a multiple of eight long, or one row, whose last block may be
// short).  Otherwise each element finds its own row and column.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(256) dropout_kernel(const DropParams p) {
    pdl_wait();
    const T* x = static_cast<const T*>(p.x);
    const T* r = static_cast<const T*>(p.r);
    T* y = static_cast<T*>(p.y);
    const int64_t total = p.rows * p.cols;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < p.blocks; b += (int64_t)gridDim.x * blockDim.x) {
        const int64_t e0 = b * 8;
        const int n = (int)min((int64_t)8, total - e0);
        if (VECTOR && n == 8) {
            constexpr int V = 16 / (int)sizeof(T), L = 8 / V;      // one load of 16-bit values, two of fp32
            int64_t row = 0, col = e0;
            if (p.rows > 1) {
                row = e0 / p.cols;
                col = e0 - row * p.cols;
            }
            const T* xr = x + row * p.xs + col;
            T* yr = y + row * p.ys + col;
            Vec<T, V> vx[L], vr[L];
#pragma unroll
            for (int l = 0; l < L; ++l) vx[l] = *reinterpret_cast<const Vec<T, V>*>(xr + l * V);
            if (r) {
#pragma unroll
                for (int l = 0; l < L; ++l)
                    vr[l] = *reinterpret_cast<const Vec<T, V>*>(r + row * p.rs + col + l * V);
            }
            const uint32_t keep = keep_bits(p, b);
#pragma unroll
            for (int l = 0; l < L; ++l) {
                float f[V], g[V];
                widen(vx[l], f);
                if (r) widen(vr[l], g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[i] = keep >> (l * V + i) & 1 ? f[i] * p.scale : 0.f;
                    if (r) f[i] += g[i];
                }
                *reinterpret_cast<Vec<T, V>*>(yr + l * V) = narrow<T, V>(f);
            }
        } else {
            const uint32_t keep = keep_bits(p, b);
            int64_t row = e0 / p.cols, col = e0 - row * p.cols;
            for (int i = 0; i < n; ++i) {
                float f = keep >> i & 1 ? to_f32(x[row * p.xs + col]) * p.scale : 0.f;
                if (r) f += to_f32(r[row * p.rs + col]);
                y[row * p.ys + col] = from_f32<T>(f);
                if (++col == p.cols) { col = 0; ++row; }
            }
        }
    }
}

template <typename T> cudaError_t run(const DropParams& p, bool vector, cudaStream_t st) {
    const int64_t most = (int64_t)device_sm_count() * 8 * 16;      // sixteen turns at most keep the tail short
    int64_t grid = (p.blocks + 255) / 256;
    if (grid > most) grid = most;
    return launch_after(vector ? dropout_kernel<T, true> : dropout_kernel<T, false>, dim3((unsigned)grid), dim3(256), 0,
                        st, p);
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
    p.none = threshold == 0;
    p.hi = (uint32_t)(threshold >> 16) & 0xffffu;
    p.lo = (uint32_t)threshold & 0xffffu;
    p.scale = d.p < 1.0 ? (float)(1.0 / (1.0 - d.p)) : 0.f;
    p.x = x; p.r = residual; p.y = y;
    const int64_t e = (int64_t)elem_bytes(d.dtype);
    const bool vector = aligned_to(x, 16) && aligned_to(y, 16) && aligned_to(residual, 16) &&
                        (flat || (d.cols % 8 == 0 && xs * e % 16 == 0 && ys * e % 16 == 0 &&
                                  (!residual || rs * e % 16 == 0)));
    switch (d.dtype) {
        case CONV2D_F32: return run<float>(p, vector, st);
        case CONV2D_F16: return run<__half>(p, vector, st);
        default: return run<__nv_bfloat16>(p, vector, st);
    }
}

}  // namespace conv2d_gb300
