// Layer norm over the channels of channels-first planes [image][channel]
// [pixel] (the layout conv2d_fwd writes), one row per pixel.
//
// x is read along pixels and y written along channels, so a block turns a tile
// of 16 words of pixels by all channels around in shared memory.  A word is
// two neighbouring pixels of a 16-bit type (when planes hold an even number of
// them), else one pixel widened to fp32; 16 words are 64 bytes of a channel's
// plane, two whole memory sectors.  A half-warp reads one channel's words; the
// 17-word pitch keeps both directions free of bank conflicts or nearly so.
// The statistics come from the tile in shared memory (mean first, then the
// squares of x - mean), so x and dy cross the memory bus once.  More channels
// than fit are taken in chunks that are read again for each step.
//
// Backward: dx needs sum a and sum a z over the channels of a pixel (a = dy
// gamma, z = (x - mean) rstd); dgamma and dbeta are sums over all pixels.
// Each warp owns 32 channels at a time; their sums over the
// tile's words are transposed-and-added across the half-warp, so one lane ends
// up with one channel, and collect in shared memory over the block's tiles.
//
// Planes of a 16-bit type with a multiple of eight pixels and of eight channels
// take a faster form (planes16_*): TMA moves tiles in and out on both sides,
// and the matrix loads and stores of shared memory (8 x 8 blocks, transposed on
// the way) hand every thread channel pairs of one pixel from either side, for
// packed arithmetic.  What bounds the general form is instructions (37 an
// element forward, 68 backward), most of them addresses.
//
// Measured, bf16, forward / backward with its sums: 64 images x 512 channels x 784
// pixels 24.6 / 41.5 us (4.2 / 3.7 TB/s) in the fast form: the tile's way through
// shared memory and its barriers hold it (issue slots 61 % busy forward, 43 %
// backward; memory 24 to 37 %).  256 x 512 x 49 pixels, general form, 22.1 / 35.6 us.
#include <cuda.h>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kWords = 16, kPitch = 17;     // words of pixels per tile, and their pitch in shared memory
// Threads of a block: few channels make small tiles, and blocks that meet less widely.
int threads_of(int C) { return C <= 128 ? 128 : 512; }

struct PlaneParams {
    int64_t rows, pixels, ys, tiles;
    int C, chunk;            // channels, and channels per chunk (a multiple of 32 unless it is all of them)
    int param_f32, pair_c;   // pair_c: y and dy rows move as pairs of 16-bit channels
    float eps, inv_c;
    const void *x, *dy, *gamma, *beta;
    void *y, *dx;
    float *mean, *rstd;
    const float *mean_in, *rstd_in;
    float* part;             // [blocks][2][C]
    int want_params;
};

// A word of PP pixels: a float, or a packed pair of 16-bit values.
template <typename T, int PP> struct Word;
template <typename T> struct Word<T, 1> {
    static __device__ __forceinline__ uint32_t load(const T* p) { return __float_as_uint(to_f32(*p)); }
    static __device__ __forceinline__ void store(T* p, uint32_t w) { *p = from_f32<T>(__uint_as_float(w)); }
    static __device__ __forceinline__ void widen(uint32_t w, float (&f)[1]) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t narrow(const float (&f)[1]) { return __float_as_uint(f[0]); }
};
template <typename T> struct Word<T, 2> {
    static __device__ __forceinline__ uint32_t load(const T* p) { return *reinterpret_cast<const uint32_t*>(p); }
    static __device__ __forceinline__ void store(T* p, uint32_t w) { *reinterpret_cast<uint32_t*>(p) = w; }
    static __device__ __forceinline__ void widen(uint32_t w, float (&f)[2]) {
        Vec<T, 2> v;
        *reinterpret_cast<uint32_t*>(&v) = w;
        conv2d_gb300::widen(v, f);
    }
    static __device__ __forceinline__ uint32_t narrow(const float (&f)[2]) {
        const Vec<T, 2> v = conv2d_gb300::narrow<T, 2>(f);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

__device__ __forceinline__ float param_at(const void* p, bool f32, bool bf16, int c, float fill) {
    if (!p) return fill;
    if (f32) return static_cast<const float*>(p)[c];
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c])
                : __half2float(static_cast<const __half*>(p)[c]);
}
template <typename T> constexpr bool is_bf16 = false;
template <> constexpr bool is_bf16<__nv_bfloat16> = true;

// Where this thread's word of a tile lies: the first pixel's offset in x
// without the channel term.
template <int PP> struct Spot {
    int64_t row, off;
    bool live;
    __device__ __forceinline__ Spot(const PlaneParams& p, int64_t tile, int word) {
        row = (tile * kWords + word) * PP;
        live = row < p.rows;
        const uint32_t n = live ? (uint32_t)row / (uint32_t)p.pixels : 0;      // both below 2^31
        off = live ? (int64_t)n * p.C * p.pixels + ((uint32_t)row - n * (uint32_t)p.pixels) : 0;
    }
};

// One chunk of x into shared memory, [channel][word].
template <typename T, int PP, int THREADS>
__device__ __forceinline__ void load_planes(const PlaneParams& p, const Spot<PP>& s, int c0, int n, int half, int word,
                                            uint32_t* tile) {
    const T* x = static_cast<const T*>(p.x) + s.off + (int64_t)c0 * p.pixels;
#pragma unroll 16
    for (int c = half; c < n; c += THREADS / 16)
        tile[c * kPitch + word] = s.live ? Word<T, PP>::load(x + c * p.pixels) : 0u;
}

// Sum of every thread's values over the channels (half-warps) of its word.
template <int PP, int THREADS>
__device__ __forceinline__ void across_halves(float (&v)[PP], int half, int word,
                                              float (*red)[THREADS / 16][kWords + 1]) {
#pragma unroll
    for (int i = 0; i < PP; ++i) red[i][half][word] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PP; ++i) {
        float s = 0.f;
#pragma unroll
        for (int h = 0; h < THREADS / 16; ++h) s += red[i][h][word];
        v[i] = s;
    }
    __syncthreads();
}

template <typename T, int PP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) planes_fwd_kernel(const PlaneParams p) {
    extern __shared__ uint32_t tile_s[];
    __shared__ float red[PP][THREADS / 16][kWords + 1];
    __shared__ float stat[2][PP][kWords];
    pdl_wait();
    const int half = threadIdx.x >> 4, word = threadIdx.x & 15;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (p.C + p.chunk - 1) / p.chunk;
    for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const Spot<PP> s(p, tile, word);
        float mean[PP], rstd[PP];
#pragma unroll
        for (int i = 0; i < PP; ++i) mean[i] = rstd[i] = 0.f;
        for (int pass = 0; pass < 2; ++pass) {
            float v[PP];
#pragma unroll
            for (int i = 0; i < PP; ++i) v[i] = 0.f;
            for (int k = 0; k < chunks; ++k) {
                const int c0 = k * p.chunk, n = min(p.chunk, p.C - c0);
                // Each thread sums the channels that it loaded itself: no barrier in between.
                if (chunks > 1 || pass == 0) load_planes<T, PP, THREADS>(p, s, c0, n, half, word, tile_s);
#pragma unroll 4
                for (int c = half; c < n; c += THREADS / 16) {
                    float f[PP];
                    Word<T, PP>::widen(tile_s[c * kPitch + word], f);
#pragma unroll
                    for (int i = 0; i < PP; ++i) {
                        if (pass == 0) v[i] += f[i];
                        else v[i] += (f[i] - mean[i]) * (f[i] - mean[i]);
                    }
                }
            }
            across_halves<PP, THREADS>(v, half, word, red);
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                if (pass == 0) mean[i] = v[i] * p.inv_c;
                else rstd[i] = rsqrtf(v[i] * p.inv_c + p.eps);
            }
        }
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                stat[0][i][word] = mean[i];
                stat[1][i][word] = rstd[i];
                if (s.live && p.mean) p.mean[s.row + i] = mean[i];
                if (s.live && p.rstd) p.rstd[s.row + i] = rstd[i];
            }
        }
        for (int k = 0; k < chunks; ++k) {
            const int c0 = k * p.chunk, n = min(p.chunk, p.C - c0);
            if (chunks > 1) {
                __syncthreads();                       // the previous chunk has been written out
                load_planes<T, PP, THREADS>(p, s, c0, n, half, word, tile_s);
            }
            __syncthreads();
            T* y = static_cast<T*>(p.y) + c0;
            if (PP == 2 && p.pair_c) {
                for (int c = 2 * lane; c < n; c += 64) {           // n is even
                    float g[2], b[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        g[i] = param_at(p.gamma, p.param_f32, is_bf16<T>, c0 + c + i, 1.f);
                        b[i] = param_at(p.beta, p.param_f32, is_bf16<T>, c0 + c + i, 0.f);
                    }
#pragma unroll
                    for (int w = warp; w < kWords; w += THREADS / 32) {
                        const int64_t row = (tile * kWords + w) * PP;
                        if (row >= p.rows) continue;
                        float f[2][PP];
                        Word<T, PP>::widen(tile_s[c * kPitch + w], f[0]);
                        Word<T, PP>::widen(tile_s[(c + 1) * kPitch + w], f[1]);
#pragma unroll
                        for (int i = 0; i < PP; ++i) {
                            const float mu = stat[0][i][w], r = stat[1][i][w];
                            const float o[2] = {(f[0][i] - mu) * r * g[0] + b[0], (f[1][i] - mu) * r * g[1] + b[1]};
                            *reinterpret_cast<Vec<T, 2>*>(y + (row + i) * p.ys + c) = narrow<T, 2>(o);
                        }
                    }
                }
            } else {
                for (int c = lane; c < n; c += 32) {
                    const float g = param_at(p.gamma, p.param_f32, is_bf16<T>, c0 + c, 1.f);
                    const float b = param_at(p.beta, p.param_f32, is_bf16<T>, c0 + c, 0.f);
#pragma unroll
                    for (int w = warp; w < kWords; w += THREADS / 32) {
                        const int64_t row = (tile * kWords + w) * PP;
                        if (row >= p.rows) continue;
                        float f[PP];
                        Word<T, PP>::widen(tile_s[c * kPitch + w], f);
#pragma unroll
                        for (int i = 0; i < PP; ++i)
                            y[(row + i) * p.ys + c] =
                                from_f32<T>((f[i] - stat[0][i][w]) * stat[1][i][w] * g + b);
                    }
                }
            }
        }
        __syncthreads();
    }
}

// One chunk of dy, read along channels, into shared memory as [channel][word].
template <typename T, int PP, int THREADS>
__device__ __forceinline__ void load_rows(const PlaneParams& p, int64_t tile, int c0, int n, int warp, int lane,
                                          uint32_t* dst) {
    const T* dy = static_cast<const T*>(p.dy) + c0;
    for (int w = warp; w < kWords; w += THREADS / 32) {
        const int64_t row = (tile * kWords + w) * PP;
        const bool live = row < p.rows;
        if constexpr (PP == 2) {
            if (p.pair_c) {
#pragma unroll 4
                for (int c = 2 * lane; c < n; c += 64) {           // n is even
                    uint32_t a = 0, b = 0;
                    if (live) {
                        a = *reinterpret_cast<const uint32_t*>(dy + row * p.ys + c);
                        b = *reinterpret_cast<const uint32_t*>(dy + (row + 1) * p.ys + c);
                    }
                    dst[c * kPitch + w] = __byte_perm(a, b, 0x5410);
                    dst[(c + 1) * kPitch + w] = __byte_perm(a, b, 0x7632);
                }
                continue;
            }
        }
#pragma unroll 4
        for (int c = lane; c < n; c += 32) {
            float f[PP];
#pragma unroll
            for (int i = 0; i < PP; ++i) f[i] = live ? to_f32(dy[(row + i) * p.ys + c]) : 0.f;
            dst[c * kPitch + w] = Word<T, PP>::narrow(f);          // widening and back is exact
        }
    }
}

template <typename T, int PP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) planes_bwd_kernel(const PlaneParams p) {
    extern __shared__ uint32_t smem[];
    __shared__ float red[PP][THREADS / 16][kWords + 1];
    const int chunks = (p.C + p.chunk - 1) / p.chunk;
    uint32_t* xs = smem;                                           // [chunk][17]
    uint32_t* ds = xs + p.chunk * kPitch;                          // [chunk][17]
    float* gam = reinterpret_cast<float*>(ds + p.chunk * kPitch);  // [C]
    float* acc = gam + p.C;                                        // [2][C]
    pdl_wait();
    const int half = threadIdx.x >> 4, word = threadIdx.x & 15;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int c = threadIdx.x; c < p.C; c += THREADS) {
        gam[c] = param_at(p.gamma, p.param_f32, is_bf16<T>, c, 1.f);
        acc[c] = acc[p.C + c] = 0.f;
    }
    __syncthreads();
    for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const Spot<PP> s(p, tile, word);
        float mu[PP], r[PP], s1[PP], s2[PP];
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            mu[i] = s.live ? p.mean_in[s.row + i] : 0.f;
            r[i] = s.live ? p.rstd_in[s.row + i] : 0.f;
            s1[i] = s2[i] = 0.f;
        }
        for (int k = 0; k < chunks; ++k) {
            const int c0 = k * p.chunk, n = min(p.chunk, p.C - c0);
            if (k > 0) __syncthreads();
            load_planes<T, PP, THREADS>(p, s, c0, n, half, word, xs);
            load_rows<T, PP, THREADS>(p, tile, c0, n, warp, lane, ds);
            __syncthreads();
#pragma unroll 4
            for (int c = half; c < n; c += THREADS / 16) {
                float fx[PP], fd[PP];
                Word<T, PP>::widen(xs[c * kPitch + word], fx);
                Word<T, PP>::widen(ds[c * kPitch + word], fd);
                const float g = gam[c0 + c];
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    const float a = fd[i] * g;
                    s1[i] += a;
                    s2[i] += a * ((fx[i] - mu[i]) * r[i]);
                }
            }
        }
        across_halves<PP, THREADS>(s1, half, word, red);
        across_halves<PP, THREADS>(s2, half, word, red);
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            s1[i] *= p.inv_c;
            s2[i] *= p.inv_c;
        }
        for (int k = 0; k < chunks; ++k) {
            const int c0 = k * p.chunk, n = min(p.chunk, p.C - c0);
            if (chunks > 1) {
                __syncthreads();
                load_planes<T, PP, THREADS>(p, s, c0, n, half, word, xs);
                load_rows<T, PP, THREADS>(p, tile, c0, n, warp, lane, ds);
                __syncthreads();
            }
            T* dx = static_cast<T*>(p.dx) + s.off + (int64_t)c0 * p.pixels;
            // A warp's 32 channels in 16 steps of two (one per half-warp).
            for (int cb = warp * 32; cb < n; cb += THREADS) {
                float vg[16], vb[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int c = cb + 2 * j + (lane >> 4);
                    vg[j] = vb[j] = 0.f;
                    if (c < n) {
                        float fx[PP], fd[PP], f[PP];
                        Word<T, PP>::widen(xs[c * kPitch + word], fx);
                        Word<T, PP>::widen(ds[c * kPitch + word], fd);
                        const float g = gam[c0 + c];
#pragma unroll
                        for (int i = 0; i < PP; ++i) {
                            const float z = (fx[i] - mu[i]) * r[i];
                            f[i] = r[i] * (fd[i] * g - s1[i] - z * s2[i]);
                            if (s.live) {
                                vg[j] += fd[i] * z;
                                vb[j] += fd[i];
                            }
                        }
                        if (p.dx && s.live) Word<T, PP>::store(dx + c * p.pixels, Word<T, PP>::narrow(f));
                    }
                }
                if (p.want_params) {
                    // Add over the 16 words while spreading the 16 steps over
                    // the lanes: after the last exchange lane l holds step l.
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) {
                        const bool up = (lane & o) != 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (j < o) {
                                const float kg = up ? vg[j + o] : vg[j], tg = up ? vg[j] : vg[j + o];
                                const float kb = up ? vb[j + o] : vb[j], tb = up ? vb[j] : vb[j + o];
                                vg[j] = kg + __shfl_xor_sync(0xffffffffu, tg, o);
                                vb[j] = kb + __shfl_xor_sync(0xffffffffu, tb, o);
                            }
                        }
                    }
                    const int c = cb + 2 * word + (lane >> 4);
                    if (c < n) {
                        acc[c0 + c] += vg[0];
                        acc[p.C + c0 + c] += vb[0];
                    }
                }
            }
        }
        __syncthreads();
    }
    if (p.want_params)
        for (int c = threadIdx.x; c < 2 * p.C; c += THREADS) p.part[(int64_t)blockIdx.x * 2 * p.C + c] = acc[c];
}

// ------------------------------------------------------------------ 16-bit, 8 x 8 blocks
// A tile is 8 PG pixels of one image by all channels, worked on by 16 warps: a
// warp takes G neighbouring groups of eight pixels of every kShares-th
// 32-channel block (NB at most), so that a channel's gamma is read once for G
// pixels.  In a block thread t has pixel t / 4 and the channel pairs
// 8 m + 2 (t % 4), m = 0..3.
//   x side   [channel][8 PG pixels]: rows of 64 or 32 bytes, as TMA writes them
//            with a swizzle of that width
//   y side   [64 channels][8 PG pixels][128 bytes], 128-byte swizzle
// so that the eight rows of a matrix lie in different banks on both sides.
constexpr int kThreads16 = 512;

template <int PG> __device__ __forceinline__ uint32_t x_at(int c, int group) {
    return (uint32_t)(c * PG * 16 + ((group ^ (c / (8 / PG) & (PG - 1))) << 4));
}
template <int PG> __device__ __forceinline__ uint32_t y_at(int pixel, int chunk) {
    return (uint32_t)((chunk >> 3) * PG * 1024 + pixel * 128 + (((chunk ^ pixel) & 7) << 4));
}

// How the 16 warps of a tile of 8 PG pixels share it, G groups of pixels each.
template <int PG, int G> struct Share {
    static constexpr int kShares = 16 * G / PG;            // warps along the channels
    int group, share;                                      // first pixel group; which share of the channel blocks
    __device__ __forceinline__ Share() {
        const int warp = threadIdx.x >> 5;
        group = warp % (PG / G) * G;
        share = warp / (PG / G);
    }
    // Pixel of group j of this thread.
    __device__ __forceinline__ int pixel(int j) const { return (group + j) * 8 + ((threadIdx.x & 31) >> 2); }
};

// N sums over a pixel's channels for each of the thread's G pixels, complete in
// every thread of the pixel: the thread's, its neighbours', then the warps'.
template <int PG, int G, int N>
__device__ __forceinline__ void pixel_sums(float (&v)[G][N], float (*red)[8 * PG][Share<PG, G>::kShares],
                                           const Share<PG, G>& sh) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[j][k] += __shfl_xor_sync(0xffffffffu, v[j][k], 1);
            v[j][k] += __shfl_xor_sync(0xffffffffu, v[j][k], 2);
            if ((threadIdx.x & 3) == 0) red[k][sh.pixel(j)][sh.share] = v[j][k];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4* q = reinterpret_cast<const float4*>(red[k][sh.pixel(j)]);
            v[j][k] = 0.f;
#pragma unroll
            for (int w = 0; w < Share<PG, G>::kShares / 4; ++w) v[j][k] += (q[w].x + q[w].y) + (q[w].z + q[w].w);
        }
    }
}

// Geometry of a launch: TMA boxes of `xbox` channels by 8 PG pixels on the x
// side, 64 channels by 8 PG pixels on the y side.
struct Boxes {
    int tpi;                 // tiles per image
    int xbox, xboxes, yboxes;
    int x_bytes, y_bytes;    // of a tile, whole boxes
};

template <int PG> __device__ __forceinline__ void load_x(const CUtensorMap* map, const Boxes& bx, int n, int px,
                                                         uint32_t dst, uint32_t bar) {
    for (int i = 0; i < bx.xboxes; ++i) tma_load_3d(dst + i * bx.xbox * PG * 16, map, bar, px, i * bx.xbox, n);
}

template <typename T, int PG, int G, int NB>
__global__ void __launch_bounds__(kThreads16, 2)
planes16_fwd_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap,
                    const PlaneParams p, const Boxes bx) {
    using S = Share<PG, G>;
    extern __shared__ uint8_t smem_raw[];                  // x side [2], y side, gamma, beta
    __shared__ __align__(16) float red[2][1][8 * PG][S::kShares];
    __shared__ uint64_t full[2];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const uint32_t xs = (smem_addr(smem_raw) + 1023u) & ~1023u, ys = xs + 2 * bx.x_bytes;
    float* gam = reinterpret_cast<float*>(smem_raw + (ys - smem_addr(smem_raw)) + bx.y_bytes);
    float* bet = gam + p.C;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&full[0]), 1);
        mbar_init(smem_addr(&full[1]), 1);
        abort_word = 0;
        mbar_fence_init();
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&ymap);
    }
    __syncthreads();
    pdl_wait();
    const S sh;
    const int lane = threadIdx.x & 31, blocks = (p.C + 31) / 32, tiles = (int)p.tiles, pixels = (int)p.pixels;
    for (int c = threadIdx.x; c < p.C; c += kThreads16) {
        gam[c] = param_at(p.gamma, p.param_f32, is_bf16<T>, c, 1.f);
        bet[c] = param_at(p.beta, p.param_f32, is_bf16<T>, c, 0.f);
    }
    auto fetch = [&](int tile, int stage) {                // (thread 0)
        const int n = (unsigned)tile / (unsigned)bx.tpi;
        mbar_arrive_expect_tx(smem_addr(&full[stage]), bx.x_bytes);
        load_x<PG>(&xmap, bx, n, (tile - n * bx.tpi) * 8 * PG, xs + stage * bx.x_bytes, smem_addr(&full[stage]));
    };
    uint32_t x_off[G][NB], y_off[G][NB];
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int b = sh.share + i * S::kShares;
            x_off[j][i] = xs + x_at<PG>(b * 32 + lane, sh.group + j);
            y_off[j][i] = ys + y_at<PG>((sh.group + j) * 8 + (lane & 7), b * 4 + (lane >> 3));
        }
    }
    int stage = 0, fetched = 0;
    uint32_t phase = 0;
    if (threadIdx.x == 0 && blockIdx.x < tiles) { fetch(blockIdx.x, 0); fetched = 1; }
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        // The tile is here, and everyone is done with the other stage.
        ok = __syncthreads_and(mbar_wait(smem_addr(&full[stage]), phase, abort_flag));
        if (!ok) break;
        if (threadIdx.x == 0 && tile + (int)gridDim.x < tiles) { fetch(tile + gridDim.x, stage ^ 1); ++fetched; }
        const uint32_t x_stage = stage * bx.x_bytes;
        f32x2 f[G][NB][4];
        float v[G][1];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            f32x2 sum = 0ull;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int b = sh.share + i * S::kShares;
                if (b < blocks) {
                    uint32_t r[4];
                    ldsm_x4_trans(x_off[j][i] + x_stage, r);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {          // (channels past C read as zero)
                        f[j][i][m] = widen_pair<T>(r[m]);
                        sum = add2(sum, f[j][i][m]);
                    }
                }
            }
            v[j][0] = sum_halves(sum);
        }
        pixel_sums<PG, G, 1>(v, red[0], sh);
        float mean[G], rstd[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            mean[j] = v[j][0] * p.inv_c;
            f32x2 sq = 0ull;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int b = sh.share + i * S::kShares;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (b * 32 + m * 8 < p.C) {
                        f[j][i][m] = add2(f[j][i][m], both(-mean[j]));
                        sq = fma2(f[j][i][m], f[j][i][m], sq);
                    }
                }
            }
            v[j][0] = sum_halves(sq);
        }
        if (threadIdx.x == 0) bulk_wait_read_all();        // the last tile's y side has been copied out
        pixel_sums<PG, G, 1>(v, red[1], sh);
        const int n = (unsigned)tile / (unsigned)bx.tpi, px = (tile - n * bx.tpi) * 8 * PG;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            rstd[j] = rsqrtf(v[j][0] * p.inv_c + p.eps);
            if (sh.share == 0 && (lane & 3) == 0 && px + sh.pixel(j) < pixels) {
                const int64_t row = (int64_t)n * pixels + px + sh.pixel(j);
                if (p.mean) p.mean[row] = mean[j];
                if (p.rstd) p.rstd[row] = rstd[j];
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int b = sh.share + i * S::kShares;
            if (b < blocks) {
                uint32_t r[G][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int c = b * 32 + m * 8 + 2 * (lane & 3);
                    if (b * 32 + m * 8 < p.C) {
                        const f32x2 g = *reinterpret_cast<const f32x2*>(gam + c);
                        const f32x2 be = *reinterpret_cast<const f32x2*>(bet + c);
#pragma unroll
                        for (int j = 0; j < G; ++j)
                            r[j][m] = narrow_pair<T>(fma2(mul2(f[j][i][m], both(rstd[j])), g, be));
                    } else {
#pragma unroll
                        for (int j = 0; j < G; ++j) r[j][m] = 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) stsm_x4(y_off[j][i], r[j]);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 0; i < bx.yboxes; ++i) tma_store_3d(&ymap, ys + i * PG * 1024, i * 64, px, n);
            bulk_commit_group();
        }
        stage ^= 1;
        if (stage == 0) phase ^= 1;
    }
    if (threadIdx.x == 0) {
        if (!ok)                                           // copies in flight land before the block leaves
            for (int i = fetched > 2 ? fetched - 2 : 0; i < fetched; ++i)
                mbar_drain_wait(smem_addr(&full[i & 1]), (uint32_t)(i >> 1) & 1u);
        bulk_wait_all();
    }
}

// dgamma and dbeta of the thread's channel pairs stay in registers over the
// block's tiles; dx goes back through the x side, whose words the same warp read.
template <typename T, int PG, int G, int NB>
__global__ void __launch_bounds__(kThreads16, NB == 1 ? 2 : 1)
planes16_bwd_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap dmap,
                    const __grid_constant__ CUtensorMap omap, const PlaneParams p, const Boxes bx) {
    using S = Share<PG, G>;
    constexpr int STAGES = 3;
    extern __shared__ uint8_t smem_raw[];                  // stages of (y side, x side), gamma
    __shared__ __align__(16) float red[2][8 * PG][S::kShares];
    __shared__ uint64_t full[STAGES];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u, stage_bytes = bx.y_bytes + bx.x_bytes;
    uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
    float* gam = reinterpret_cast<float*>(smem + STAGES * stage_bytes);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(smem_addr(&full[i]), 1);
        abort_word = 0;
        mbar_fence_init();
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&dmap);
    }
    __syncthreads();
    pdl_wait();
    const S sh;
    const int lane = threadIdx.x & 31, blocks = (p.C + 31) / 32, tiles = (int)p.tiles, pixels = (int)p.pixels;
    for (int c = threadIdx.x; c < p.C; c += kThreads16) gam[c] = param_at(p.gamma, p.param_f32, is_bf16<T>, c, 1.f);
    auto fetch = [&](int tile, int stage) {                // (thread 0)
        const uint32_t bar = smem_addr(&full[stage]), dst = base + stage * stage_bytes;
        const int n = (unsigned)tile / (unsigned)bx.tpi, px = (tile - n * bx.tpi) * 8 * PG;
        mbar_arrive_expect_tx(bar, stage_bytes);
        for (int i = 0; i < bx.yboxes; ++i) tma_load_3d(dst + i * PG * 1024, &dmap, bar, i * 64, px, n);
        load_x<PG>(&xmap, bx, n, px, dst + bx.y_bytes, bar);
    };
    uint32_t x_off[G][NB], d_off[G][NB];
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int b = sh.share + i * S::kShares;
            d_off[j][i] = base + y_at<PG>((sh.group + j) * 8 + (lane & 7), b * 4 + (lane >> 3));
            x_off[j][i] = base + bx.y_bytes + x_at<PG>(b * 32 + lane, sh.group + j);
        }
    }
    f32x2 dg[NB][4], db[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) dg[i][m] = db[i][m] = 0ull;
    int fetched = 0, stage = 0;
    uint32_t phase = 0;
    if (threadIdx.x == 0)
        for (int t = blockIdx.x; fetched < STAGES - 1 && t < tiles; t += gridDim.x, ++fetched) fetch(t, fetched);
    // Statistics of the thread's pixels; past the image both are zero, which
    // makes every term of the tile's empty pixels zero (their x and dy are).
    float nmu[G], nr[G];
    auto stats = [&](int tile) {
        const int n = (unsigned)tile / (unsigned)bx.tpi, px = (tile - n * bx.tpi) * 8 * PG;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            nmu[j] = nr[j] = 0.f;
            if (tile < tiles && px + sh.pixel(j) < pixels) {
                nmu[j] = p.mean_in[(int64_t)n * pixels + px + sh.pixel(j)];
                nr[j] = p.rstd_in[(int64_t)n * pixels + px + sh.pixel(j)];
            }
        }
    };
    stats(blockIdx.x);
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        float mu[G], r[G];
#pragma unroll
        for (int j = 0; j < G; ++j) { mu[j] = nmu[j]; r[j] = nr[j]; }
        stats(tile + gridDim.x);
        // The tile is here; the last one's dx, whose stage is next, has been copied out.
        bool landed = mbar_wait(smem_addr(&full[stage]), phase, abort_flag);
        if (threadIdx.x == 0) bulk_wait_read_all();
        ok = __syncthreads_and(landed);
        if (!ok) break;
        if (threadIdx.x == 0 && tile + (STAGES - 1) * (int)gridDim.x < tiles) {
            fetch(tile + (STAGES - 1) * gridDim.x, stage == 0 ? STAGES - 1 : stage - 1);
            ++fetched;
        }
        const uint32_t at = stage * stage_bytes;
        f32x2 s1[G], s2[G];
#pragma unroll
        for (int j = 0; j < G; ++j) s1[j] = s2[j] = 0ull;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int b = sh.share + i * S::kShares;
            if (b < blocks) {
                uint32_t rx[G][4], rd[G][4];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    ldsm_x4_trans(x_off[j][i] + at, rx[j]);
                    ldsm_x4(d_off[j][i] + at, rd[j]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (b * 32 + m * 8 < p.C) {            // with u = dy (x - mean): a z = gamma u r, dy z = u r
                        const f32x2 g = *reinterpret_cast<const f32x2*>(gam + b * 32 + m * 8 + 2 * (lane & 3));
#pragma unroll
                        for (int j = 0; j < G; ++j) {
                            const f32x2 d = widen_pair<T>(rd[j][m]);
                            const f32x2 u = mul2(d, add2(widen_pair<T>(rx[j][m]), both(-mu[j])));
                            s1[j] = fma2(d, g, s1[j]);
                            s2[j] = fma2(u, g, s2[j]);
                            dg[i][m] = fma2(u, both(r[j]), dg[i][m]);
                            db[i][m] = add2(db[i][m], d);
                        }
                    }
                }
            }
        }
        if (p.dx) {
            float v[G][2];
            f32x2 n1[G], n2[G];
#pragma unroll
            for (int j = 0; j < G; ++j) { v[j][0] = sum_halves(s1[j]); v[j][1] = sum_halves(s2[j]); }
            pixel_sums<PG, G, 2>(v, red, sh);
#pragma unroll
            for (int j = 0; j < G; ++j) {                  // dx = r a - r mean(a) - (x - mean) r^3 mean(gamma u)
                n1[j] = both(-v[j][0] * p.inv_c * r[j]);
                n2[j] = both(-v[j][1] * p.inv_c * r[j] * r[j] * r[j]);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int b = sh.share + i * S::kShares;
                if (b < blocks) {
                    uint32_t rx[G][4], rd[G][4];
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        ldsm_x4_trans(x_off[j][i] + at, rx[j]);
                        ldsm_x4(d_off[j][i] + at, rd[j]);
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        if (b * 32 + m * 8 < p.C) {
                            const f32x2 g = *reinterpret_cast<const f32x2*>(gam + b * 32 + m * 8 + 2 * (lane & 3));
#pragma unroll
                            for (int j = 0; j < G; ++j)
                                rx[j][m] = narrow_pair<T>(
                                    fma2(mul2(widen_pair<T>(rd[j][m]), g), both(r[j]),
                                         fma2(add2(widen_pair<T>(rx[j][m]), both(-mu[j])), n2[j], n1[j])));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < G; ++j) stsm_x4_trans(x_off[j][i] + at, rx[j]);
                }
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (threadIdx.x == 0) {
                const int n = (unsigned)tile / (unsigned)bx.tpi, px = (tile - n * bx.tpi) * 8 * PG;
                for (int i = 0; i < bx.xboxes; ++i)
                    tma_store_3d(&omap, base + at + bx.y_bytes + i * bx.xbox * PG * 16, px, i * bx.xbox, n);
                bulk_commit_group();
            }
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
    }
    if (threadIdx.x == 0) {
        if (!ok)                                           // copies in flight land before the block leaves
            for (int i = fetched > STAGES ? fetched - STAGES : 0; i < fetched; ++i)
                mbar_drain_wait(smem_addr(&full[i % STAGES]), (uint32_t)(i / STAGES) & 1u);
        bulk_wait_all();
    }
    if (!p.want_params) return;
    // Add the eight pixels of a matrix (every exchange halves the values that a
    // lane carries: value 4 m + 2 q + e, channel pair m, dgamma or dbeta q, ends
    // up in the lanes with m in bits 3-4 and q in bit 2), then the warps that
    // share a channel block.
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);           // [pixel group share][2][channels of the blocks]
    const int width = blocks * 32;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int b = sh.share + i * S::kShares;
        float v[16];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            unpack2f(dg[i][m], v[4 * m], v[4 * m + 1]);
            unpack2f(db[i][m], v[4 * m + 2], v[4 * m + 3]);
        }
        int o = 16;
#pragma unroll
        for (int n = 8; n > 1; n >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int k = 0; k < n; ++k)
                v[k] = (up ? v[k + n] : v[k]) + __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + n], o);
        }
        if (b < blocks) {
            const int m = lane >> 3, q = lane >> 2 & 1;
            float* dst = acc + ((sh.group / G) * 2 + q) * width + b * 32 + m * 8 + 2 * (lane & 3);
            dst[0] = v[0];
            dst[1] = v[1];
        }
    }
    __syncthreads();
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.C;
    for (int c = threadIdx.x; c < p.C; c += kThreads16) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float u = acc[q * width + c];
#pragma unroll
            for (int k = 1; k < PG / G; ++k) u += acc[(2 * k + q) * width + c];
            out[q * p.C + c] = u;
        }
    }
}

constexpr int kSmemMost = 200 * 1024;     // (no form asks for more: the fast backward with 1024 channels takes 197 KB)

int chunk_of(int C, int tiles_held, int other_bytes) {
    const int64_t most = (kSmemMost - other_bytes) / (tiles_held * kPitch * 4);
    if (C <= most) return C;
    return (int)(most / 32 * 32);
}

template <typename T, int PP, int THREADS>
cudaError_t fwd_planes_at(PlaneParams p, cudaStream_t st) {
    p.tiles = (p.rows + kWords * PP - 1) / (kWords * PP);
    p.chunk = chunk_of(p.C, 1, 0);
    const int smem = p.chunk * kPitch * 4;
    const cudaError_t e = allow_smem(planes_fwd_kernel<T, PP, THREADS>, kSmemMost);
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)device_sm_count() * (2048 / THREADS);
    if (grid > p.tiles) grid = p.tiles;
    return launch_after(planes_fwd_kernel<T, PP, THREADS>, dim3((unsigned)grid), dim3(THREADS), smem, st, p);
}

template <typename T, int PP> cudaError_t fwd_planes(const PlaneParams& p, cudaStream_t st) {
    return threads_of(p.C) == 128 ? fwd_planes_at<T, PP, 128>(p, st) : fwd_planes_at<T, PP, 512>(p, st);
}

template <typename T, int PP, int THREADS>
cudaError_t bwd_planes_at(PlaneParams p, int* parts, cudaStream_t st) {
    p.tiles = (p.rows + kWords * PP - 1) / (kWords * PP);
    p.chunk = chunk_of(p.C, 2, 3 * p.C * 4);
    const int smem = 2 * p.chunk * kPitch * 4 + 3 * p.C * 4;
    const cudaError_t e = allow_smem(planes_bwd_kernel<T, PP, THREADS>, kSmemMost);
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)device_sm_count() * (1024 / THREADS);
    if (grid > p.tiles) grid = p.tiles;
    *parts = (int)grid;
    return launch_after(planes_bwd_kernel<T, PP, THREADS>, dim3((unsigned)grid), dim3(THREADS), smem, st, p);
}

// Whether the 16-bit form serves the call: what TMA moves starts and repeats at
// 16-byte boundaries, and 16 warps hold all channels.
bool fast16(const layernorm_desc& d, const void* x, const void* dx, const void* rows) {
    return d.dtype != CONV2D_F32 && d.pixels % 8 == 0 && d.cols % 8 == 0 && d.cols <= 1024 && d.ys % 8 == 0 &&
           aligned_to(x, 16) && aligned_to(dx, 16) && aligned_to(rows, 16) && d.ys < (1LL << 38);
}

typedef CUresult (*PFN_encode_t)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A 3-D 16-bit tensor (innermost first), boxes of b0 x b1 x 1, zeros outside.
bool map3(CUtensorMap* m, const void* base, bool bf16, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2,
          int b0, int b1, CUtensorMapSwizzle swizzle) {
    static PFN_encode_t enc = reinterpret_cast<PFN_encode_t>(driver_entry("cuTensorMapEncodeTiled"));
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t str[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
    cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, 1}, es[3] = {1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void*>(base), dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PG> Boxes boxes_of(PlaneParams& p) {
    Boxes b;
    b.tpi = (int)((p.pixels + 8 * PG - 1) / (8 * PG));
    p.tiles = p.rows / p.pixels * b.tpi;
    const int c32 = (p.C + 31) / 32 * 32;
    b.xbox = c32 < 256 ? c32 : 256;
    b.xboxes = (p.C + b.xbox - 1) / b.xbox;
    b.yboxes = (p.C + 63) / 64;
    b.x_bytes = (b.xboxes * b.xbox * PG * 16 + 1023) / 1024 * 1024;
    b.y_bytes = b.yboxes * PG * 1024;
    return b;
}
template <int PG> bool x_map(CUtensorMap* m, const PlaneParams& p, const Boxes& b, const void* x, bool bf16) {
    return map3(m, x, bf16, p.pixels, p.C, p.rows / p.pixels, p.pixels, p.pixels * p.C, 8 * PG, b.xbox,
                PG == 4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
}
template <int PG> bool y_map(CUtensorMap* m, const PlaneParams& p, const void* y, bool bf16) {
    return map3(m, y, bf16, p.C, p.pixels, p.rows / p.pixels, p.ys, p.ys * p.pixels, 64, 8 * PG,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int PG, int G, int NB> cudaError_t fwd_fast(PlaneParams p, cudaStream_t st) {
    const Boxes b = boxes_of<PG>(p);
    CUtensorMap xm, ym;
    if (!x_map<PG>(&xm, p, b, p.x, is_bf16<T>) || !y_map<PG>(&ym, p, p.y, is_bf16<T>)) return cudaErrorInvalidValue;
    const int smem = 1024 + 2 * b.x_bytes + b.y_bytes + 2 * p.C * 4;
    const cudaError_t e = allow_smem(planes16_fwd_kernel<T, PG, G, NB>, kSmemMost);
    if (e != cudaSuccess) return e;
    int64_t grid = 2 * device_sm_count();
    if (grid > p.tiles) grid = p.tiles;
    return launch_after(planes16_fwd_kernel<T, PG, G, NB>, dim3((unsigned)grid), dim3(kThreads16), smem, st, xm, ym, p,
                        b);
}

template <typename T, int PG, int G, int NB> cudaError_t bwd_fast(PlaneParams p, int* parts, cudaStream_t st) {
    const Boxes b = boxes_of<PG>(p);
    CUtensorMap xm, dm, om;
    if (!x_map<PG>(&xm, p, b, p.x, is_bf16<T>) || !y_map<PG>(&dm, p, p.dy, is_bf16<T>) ||
        !x_map<PG>(&om, p, b, p.dx ? p.dx : p.x, is_bf16<T>))
        return cudaErrorInvalidValue;
    const int smem = 1024 + 3 * (b.x_bytes + b.y_bytes) + p.C * 4;
    const cudaError_t e = allow_smem(planes16_bwd_kernel<T, PG, G, NB>, kSmemMost);
    if (e != cudaSuccess) return e;
    int64_t grid = device_sm_count() * (NB == 1 ? 2 : 1);
    if (grid > p.tiles) grid = p.tiles;
    *parts = (int)grid;
    return launch_after(planes16_bwd_kernel<T, PG, G, NB>, dim3((unsigned)grid), dim3(kThreads16), smem, st, xm, dm, om,
                        p, b);
}

// Tiles of 32 pixels up to 512 channels (64-byte runs of a plane), 16 beyond.
template <typename T> cudaError_t fwd_16(const PlaneParams& p, cudaStream_t st) {
    if (p.C <= 128) return fwd_fast<T, 4, 1, 1>(p, st);
    if (p.C <= 256) return fwd_fast<T, 4, 2, 1>(p, st);
    if (p.C <= 512) return fwd_fast<T, 4, 2, 2>(p, st);
    return fwd_fast<T, 2, 2, 2>(p, st);
}
template <typename T> cudaError_t bwd_16(const PlaneParams& p, int* parts, cudaStream_t st) {
    if (p.C <= 128) return bwd_fast<T, 4, 1, 1>(p, parts, st);
    if (p.C <= 256) return bwd_fast<T, 4, 2, 1>(p, parts, st);
    if (p.C <= 512) return bwd_fast<T, 4, 2, 2>(p, parts, st);
    return bwd_fast<T, 2, 2, 2>(p, parts, st);
}

template <typename T, int PP> cudaError_t bwd_planes(const PlaneParams& p, int* parts, cudaStream_t st) {
    return threads_of(p.C) == 128 ? bwd_planes_at<T, PP, 128>(p, parts, st) : bwd_planes_at<T, PP, 512>(p, parts, st);
}

PlaneParams params_of(const layernorm_desc& d) {
    PlaneParams p{};
    p.rows = d.rows; p.pixels = d.pixels; p.ys = d.ys; p.C = (int)d.cols;
    p.param_f32 = d.param == CONV2D_F32;
    p.eps = d.eps;
    p.inv_c = 1.0f / (float)d.cols;
    return p;
}

// Pixel pairs need 4-byte aligned planes, channel pairs 4-byte aligned rows.
bool pair_pixels(const layernorm_desc& d, const void* a, const void* b) {
    return d.dtype != CONV2D_F32 && d.pixels % 2 == 0 && aligned_to(a, 4) && aligned_to(b, 4);
}
bool pair_channels(const layernorm_desc& d, const void* r) {
    return d.cols % 2 == 0 && d.ys % 2 == 0 && aligned_to(r, 4);
}

}  // namespace

cudaError_t status_word_lp(void** p) { return unit_status_word(p); }
cudaError_t wait_limit_set_lp(cudaStream_t st, uint64_t ns) { return unit_wait_limit_set(st, ns); }

cudaError_t launch_layernorm_planes_fwd(const layernorm_desc& d, const void* x, const void* gamma, const void* beta,
                                        void* y, float* mean, float* rstd, cudaStream_t st) {
    PlaneParams p = params_of(d);
    p.x = x; p.gamma = gamma; p.beta = beta; p.y = y; p.mean = mean; p.rstd = rstd;
    if (fast16(d, x, nullptr, y))
        return d.dtype == CONV2D_F16 ? fwd_16<__half>(p, st) : fwd_16<__nv_bfloat16>(p, st);
    p.pair_c = pair_channels(d, y);
    const bool pair = pair_pixels(d, x, x);
    switch (d.dtype) {
        case CONV2D_F32: return fwd_planes<float, 1>(p, st);
        case CONV2D_F16: return pair ? fwd_planes<__half, 2>(p, st) : fwd_planes<__half, 1>(p, st);
        default: return pair ? fwd_planes<__nv_bfloat16, 2>(p, st) : fwd_planes<__nv_bfloat16, 1>(p, st);
    }
}

size_t layernorm_planes_bwd_workspace(const layernorm_desc& d) {
    return (size_t)device_sm_count() * (1024 / threads_of((int)d.cols)) * 2 * (size_t)d.cols * sizeof(float);
}

cudaError_t launch_layernorm_planes_bwd(const layernorm_desc& d, const void* dy, const void* x, const void* gamma,
                                        const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                                        void* ws, cudaStream_t st) {
    PlaneParams p = params_of(d);
    p.x = x; p.dy = dy; p.gamma = gamma; p.dx = dx; p.mean_in = mean; p.rstd_in = rstd;
    p.part = static_cast<float*>(ws);
    p.want_params = dgamma || dbeta;
    p.pair_c = pair_channels(d, dy);
    const bool pair = pair_pixels(d, x, dx);
    int parts = 0;
    cudaError_t e;
    if (fast16(d, x, dx, dy)) {
        e = d.dtype == CONV2D_F16 ? bwd_16<__half>(p, &parts, st) : bwd_16<__nv_bfloat16>(p, &parts, st);
    } else switch (d.dtype) {
        case CONV2D_F32: e = bwd_planes<float, 1>(p, &parts, st); break;
        case CONV2D_F16: e = pair ? bwd_planes<__half, 2>(p, &parts, st) : bwd_planes<__half, 1>(p, &parts, st); break;
        default: e = pair ? bwd_planes<__nv_bfloat16, 2>(p, &parts, st) : bwd_planes<__nv_bfloat16, 1>(p, &parts, st);
    }
    if (e != cudaSuccess || !p.want_params) return e;
    return launch_layernorm_params(p.part, parts, d, dgamma, dbeta, st);
}

}  // namespace conv2d_gb300
