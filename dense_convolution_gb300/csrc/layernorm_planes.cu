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
// Each warp owns 32 channels of a 512-channel step; their sums over the
// tile's words are transposed-and-added across the half-warp, so one lane ends
// up with one channel, and collect in shared memory over the block's tiles.
//
// Planes of a 16-bit type with a multiple of four pixels and of eight channels
// (every 16-bit layer of this library's workloads) take a faster form
// (planes16_*): a thread holds two channels by four pixels, so a load or store
// moves four pixels (or, in shared memory, a channel pair) and the index
// arithmetic is shared by eight elements.  The general form spends 37
// instructions an element forward and 68 backward, which bounds it.
#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kWords = 16, kPitch = 17;     // words of pixels per tile, and their pitch in shared memory
constexpr int kFwdThreads = 256, kBwdThreads = 512;

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
        const int64_t n = live ? row / p.pixels : 0;
        off = live ? n * p.C * p.pixels + (row - n * p.pixels) : 0;
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

template <typename T, int PP>
__global__ void __launch_bounds__(kFwdThreads, 4) planes_fwd_kernel(const PlaneParams p) {
    extern __shared__ uint32_t tile_s[];
    __shared__ float red[PP][kFwdThreads / 16][kWords + 1];
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
                if (chunks > 1 || pass == 0) load_planes<T, PP, kFwdThreads>(p, s, c0, n, half, word, tile_s);
#pragma unroll 4
                for (int c = half; c < n; c += kFwdThreads / 16) {
                    float f[PP];
                    Word<T, PP>::widen(tile_s[c * kPitch + word], f);
#pragma unroll
                    for (int i = 0; i < PP; ++i) {
                        if (pass == 0) v[i] += f[i];
                        else v[i] += (f[i] - mean[i]) * (f[i] - mean[i]);
                    }
                }
            }
            across_halves<PP, kFwdThreads>(v, half, word, red);
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                if (pass == 0) mean[i] = v[i] * p.inv_c;
                else rstd[i] = 1.0f / sqrtf(v[i] * p.inv_c + p.eps);
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
                load_planes<T, PP, kFwdThreads>(p, s, c0, n, half, word, tile_s);
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
                    for (int w = warp; w < kWords; w += kFwdThreads / 32) {
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
                    for (int w = warp; w < kWords; w += kFwdThreads / 32) {
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
template <typename T, int PP>
__device__ __forceinline__ void load_rows(const PlaneParams& p, int64_t tile, int c0, int n, int warp, int lane,
                                          uint32_t* dst) {
    const T* dy = static_cast<const T*>(p.dy) + c0;
    for (int w = warp; w < kWords; w += kBwdThreads / 32) {
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

template <typename T, int PP>
__global__ void __launch_bounds__(kBwdThreads, 2) planes_bwd_kernel(const PlaneParams p) {
    extern __shared__ uint32_t smem[];
    __shared__ float red[PP][kBwdThreads / 16][kWords + 1];
    const int chunks = (p.C + p.chunk - 1) / p.chunk;
    uint32_t* xs = smem;                                           // [chunk][17]
    uint32_t* ds = xs + p.chunk * kPitch;                          // [chunk][17]
    float* gam = reinterpret_cast<float*>(ds + p.chunk * kPitch);  // [C]
    float* acc = gam + p.C;                                        // [2][C]
    pdl_wait();
    const int half = threadIdx.x >> 4, word = threadIdx.x & 15;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int c = threadIdx.x; c < p.C; c += kBwdThreads) {
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
            load_planes<T, PP, kBwdThreads>(p, s, c0, n, half, word, xs);
            load_rows<T, PP>(p, tile, c0, n, warp, lane, ds);
            __syncthreads();
#pragma unroll 4
            for (int c = half; c < n; c += kBwdThreads / 16) {
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
        across_halves<PP, kBwdThreads>(s1, half, word, red);
        across_halves<PP, kBwdThreads>(s2, half, word, red);
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            s1[i] *= p.inv_c;
            s2[i] *= p.inv_c;
        }
        for (int k = 0; k < chunks; ++k) {
            const int c0 = k * p.chunk, n = min(p.chunk, p.C - c0);
            if (chunks > 1) {
                __syncthreads();
                load_planes<T, PP, kBwdThreads>(p, s, c0, n, half, word, xs);
                load_rows<T, PP>(p, tile, c0, n, warp, lane, ds);
                __syncthreads();
            }
            T* dx = static_cast<T*>(p.dx) + s.off + (int64_t)c0 * p.pixels;
            // A warp's 32 channels in 16 steps of two (one per half-warp).
            for (int cb = warp * 32; cb < n; cb += kBwdThreads) {
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
        for (int c = threadIdx.x; c < 2 * p.C; c += kBwdThreads) p.part[(int64_t)blockIdx.x * 2 * p.C + c] = acc[c];
}

// ------------------------------------------------------------------ 16-bit, four pixels a thread
// A tile is 32 pixels by all channels.  Lane l & 7 of a warp holds pixels
// 4 l .. 4 l + 3, lane >> 3 (and the warp) the channel pair.  The [pixel]
// [channel] side of the tile sits in shared memory in 16-byte chunks of eight
// channels, chunk k of pixel q at k ^ (q / 4 % 8): eight lanes of different
// pixels then meet different banks, and so do a row's consecutive chunks.
constexpr int kTile = 32;

__device__ __forceinline__ uint32_t chunk_at(int pixel, int chunk, int pitch) {
    return (uint32_t)(pixel * pitch * 2 + ((chunk ^ (pixel >> 2 & 7)) << 4));
}
template <typename T> __device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
    float f[2];
    Word<T, 2>::widen(w, f);
    a = f[0];
    b = f[1];
}
template <typename T> __device__ __forceinline__ void widen4(uint2 w, float (&f)[4]) {
    widen2<T>(w.x, f[0], f[1]);
    widen2<T>(w.y, f[2], f[3]);
}
template <typename T> __device__ __forceinline__ uint32_t pair(float a, float b) {
    const float f[2] = {a, b};
    return Word<T, 2>::narrow(f);
}

template <typename T, int NP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) planes16_fwd_kernel(const PlaneParams p) {
    extern __shared__ __align__(16) uint8_t tile_b[];
    __shared__ float4 red[2][THREADS / 32][8];
    pdl_wait();
    const int l = threadIdx.x & 7, k0 = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = (p.C + 63) / 64 * 64;
    const int64_t tile = blockIdx.x, row0 = tile * kTile + 4 * l;
    const bool live = row0 < p.rows;
    const int64_t n = live ? row0 / p.pixels : 0, off = live ? n * p.C * p.pixels + (row0 - n * p.pixels) : 0;
    const T* x = static_cast<const T*>(p.x) + off;
    uint2 raw[NP][2];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int c = 2 * (k0 + j * (THREADS / 8));
        raw[j][0] = raw[j][1] = make_uint2(0, 0);
        if (live && c < p.C) {
            raw[j][0] = *reinterpret_cast<const uint2*>(x + c * p.pixels);
            raw[j][1] = *reinterpret_cast<const uint2*>(x + (c + 1) * p.pixels);
        }
    }
    // Sum over the channels: this thread's, the warp's four pairs, the warps.
    auto total = [&](float (&v)[4], int which) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
        }
        if (lane < 8) red[which][warp][l] = make_float4(v[0], v[1], v[2], v[3]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            const float4 t = red[which][w][l];
            v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= p.inv_c;
    };
    float mean[4] = {0.f, 0.f, 0.f, 0.f}, rstd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float f[4];
            widen4<T>(raw[j][e], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) mean[i] += f[i];
        }
    }
    total(mean, 0);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        if (2 * (k0 + j * (THREADS / 8)) < p.C) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f[4];
                widen4<T>(raw[j][e], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) rstd[i] += (f[i] - mean[i]) * (f[i] - mean[i]);
            }
        }
    }
    total(rstd, 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) rstd[i] = 1.0f / sqrtf(rstd[i] + p.eps);
    if (threadIdx.x < 8 && live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p.mean) p.mean[row0 + i] = mean[i];
            if (p.rstd) p.rstd[row0 + i] = rstd[i];
        }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int c = 2 * (k0 + j * (THREADS / 8));
        if (c < p.C) {
            const float g0 = param_at(p.gamma, p.param_f32, is_bf16<T>, c, 1.f);
            const float g1 = param_at(p.gamma, p.param_f32, is_bf16<T>, c + 1, 1.f);
            const float b0 = param_at(p.beta, p.param_f32, is_bf16<T>, c, 0.f);
            const float b1 = param_at(p.beta, p.param_f32, is_bf16<T>, c + 1, 0.f);
            float f0[4], f1[4];
            widen4<T>(raw[j][0], f0);
            widen4<T>(raw[j][1], f1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint32_t*>(tile_b + chunk_at(4 * l + i, c >> 3, pitch) + (c & 7) * 2) =
                    pair<T>((f0[i] - mean[i]) * rstd[i] * g0 + b0, (f1[i] - mean[i]) * rstd[i] * g1 + b1);
        }
    }
    __syncthreads();
    for (int q = warp; q < kTile; q += THREADS / 32) {
        const int64_t row = tile * kTile + q;
        if (row >= p.rows) break;
        T* y = static_cast<T*>(p.y) + row * p.ys;
        for (int k = lane; k < p.C / 8; k += 32)
            *reinterpret_cast<uint4*>(y + k * 8) = *reinterpret_cast<const uint4*>(tile_b + chunk_at(q, k, pitch));
    }
}

__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One block of 512 threads per SM (two for few channels) over many tiles.
// Asynchronous copies bring later tiles in while this one is worked on: x into
// the thread's own words, dy into the swizzled tile.  dgamma and dbeta of the
// thread's channels stay in registers until the end.
template <typename T, int NP>
__global__ void __launch_bounds__(512, NP <= 2 ? 2 : 1) planes16_bwd_kernel(const PlaneParams p) {
    constexpr int STAGES = NP == 8 ? 1 : 3, XBYTES = NP * 8192;
    extern __shared__ __align__(16) uint8_t smem_b[];
    __shared__ float4 red[2][16][8];
    pdl_wait();
    const int l = threadIdx.x & 7, k0 = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = (p.C + 63) / 64 * 64, stage_bytes = XBYTES + kTile * pitch * 2;
    float* gam = reinterpret_cast<float*>(smem_b + STAGES * stage_bytes);
    for (int c = threadIdx.x; c < p.C; c += 512) gam[c] = param_at(p.gamma, p.param_f32, is_bf16<T>, c, 1.f);

    auto place = [&](int64_t tile, int64_t& row0) {        // offset of this thread's pixels, or -1
        row0 = tile * kTile + 4 * l;
        if (row0 >= p.rows) return (int64_t)-1;
        const int64_t n = row0 / p.pixels;
        return n * p.C * p.pixels + (row0 - n * p.pixels);
    };
    auto issue = [&](int64_t tile, int stage) {
        int64_t row0;
        const int64_t off = tile < p.tiles ? place(tile, row0) : -1;
        const uint32_t xd = smem_addr(smem_b + stage * stage_bytes) + threadIdx.x * 8;
        if (off >= 0) {
            const T* x = static_cast<const T*>(p.x) + off;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int c = 2 * (k0 + j * 64);
                if (c < p.C) {
                    copy_async8(xd + j * 8192, x + c * p.pixels);
                    copy_async8(xd + j * 8192 + 4096, x + (c + 1) * p.pixels);
                }
            }
        }
        if (tile < p.tiles) {
            const uint32_t dd = smem_addr(smem_b + stage * stage_bytes) + XBYTES;
#pragma unroll
            for (int q = warp; q < kTile; q += 16) {
                const int64_t row = tile * kTile + q;
                if (row < p.rows) {
                    const T* dy = static_cast<const T*>(p.dy) + row * p.ys;
                    for (int k = lane; k < p.C / 8; k += 32) copy_async16(dd + chunk_at(q, k, pitch), dy + k * 8);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    float ag[NP][2], ab[NP][2];
#pragma unroll
    for (int j = 0; j < NP; ++j) ag[j][0] = ag[j][1] = ab[j][0] = ab[j][1] = 0.f;
    float nmu[4], nr[4];
    auto stats = [&](int64_t tile) {
        int64_t row0;
        const bool live = tile < p.tiles && place(tile, row0) >= 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nmu[i] = live ? p.mean_in[row0 + i] : 0.f;
            nr[i] = live ? p.rstd_in[row0 + i] : 0.f;
        }
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(blockIdx.x + (int64_t)s * gridDim.x, s);
    stats(blockIdx.x);
    int stage = 0;
    for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int ahead = STAGES == 1 ? 0 : (stage == 0 ? STAGES - 1 : stage - 1);
        issue(tile + (int64_t)(STAGES - 1) * gridDim.x, ahead);
        float mu[4], r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { mu[i] = nmu[i]; r[i] = nr[i]; }
        stats(tile + gridDim.x);
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncthreads();
        int64_t row0;
        const int64_t off = place(tile, row0);
        const uint8_t* xs = smem_b + stage * stage_bytes + threadIdx.x * 8;
        const uint8_t* ds = smem_b + stage * stage_bytes + XBYTES;
        float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        if (off >= 0) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int c = 2 * (k0 + j * 64);
                if (c < p.C) {
                    float x0[4], x1[4];
                    widen4<T>(*reinterpret_cast<const uint2*>(xs + j * 8192), x0);
                    widen4<T>(*reinterpret_cast<const uint2*>(xs + j * 8192 + 4096), x1);
                    const float2 g = *reinterpret_cast<const float2*>(gam + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float d0, d1;
                        widen2<T>(*reinterpret_cast<const uint32_t*>(ds + chunk_at(4 * l + i, c >> 3, pitch) + (c & 7) * 2),
                                  d0, d1);
                        const float z0 = (x0[i] - mu[i]) * r[i], z1 = (x1[i] - mu[i]) * r[i];
                        const float a0 = d0 * g.x, a1 = d1 * g.y;
                        s1[i] += a0 + a1;
                        s2[i] = fmaf(a0, z0, fmaf(a1, z1, s2[i]));
                        ag[j][0] = fmaf(d0, z0, ag[j][0]);
                        ag[j][1] = fmaf(d1, z1, ag[j][1]);
                        ab[j][0] += d0;
                        ab[j][1] += d1;
                    }
                }
            }
        }
        if (p.dx) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s1[i] += __shfl_xor_sync(0xffffffffu, s1[i], 8);
                s2[i] += __shfl_xor_sync(0xffffffffu, s2[i], 8);
                s1[i] += __shfl_xor_sync(0xffffffffu, s1[i], 16);
                s2[i] += __shfl_xor_sync(0xffffffffu, s2[i], 16);
            }
            if (lane < 8) {
                red[0][warp][l] = make_float4(s1[0], s1[1], s1[2], s1[3]);
                red[1][warp][l] = make_float4(s2[0], s2[1], s2[2], s2[3]);
            }
            __syncthreads();
            if (off >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s1[i] = s2[i] = 0.f;
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    const float4 a = red[0][w][l], b = red[1][w][l];
                    s1[0] += a.x; s1[1] += a.y; s1[2] += a.z; s1[3] += a.w;
                    s2[0] += b.x; s2[1] += b.y; s2[2] += b.z; s2[3] += b.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {              // dx = r a - r s1 - (x - mu) r r s2
                    s1[i] *= p.inv_c * r[i];
                    s2[i] *= p.inv_c * r[i] * r[i];
                }
                T* dx = static_cast<T*>(p.dx) + off;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const int c = 2 * (k0 + j * 64);
                    if (c < p.C) {
                        float x0[4], x1[4];
                        widen4<T>(*reinterpret_cast<const uint2*>(xs + j * 8192), x0);
                        widen4<T>(*reinterpret_cast<const uint2*>(xs + j * 8192 + 4096), x1);
                        const float2 g = *reinterpret_cast<const float2*>(gam + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float d0, d1;
                            widen2<T>(*reinterpret_cast<const uint32_t*>(ds + chunk_at(4 * l + i, c >> 3, pitch) +
                                                                         (c & 7) * 2), d0, d1);
                            x0[i] = fmaf(d0 * g.x, r[i], -fmaf(x0[i] - mu[i], s2[i], s1[i]));
                            x1[i] = fmaf(d1 * g.y, r[i], -fmaf(x1[i] - mu[i], s2[i], s1[i]));
                        }
                        *reinterpret_cast<uint2*>(dx + c * p.pixels) =
                            make_uint2(pair<T>(x0[0], x0[1]), pair<T>(x0[2], x0[3]));
                        *reinterpret_cast<uint2*>(dx + (c + 1) * p.pixels) =
                            make_uint2(pair<T>(x1[0], x1[1]), pair<T>(x1[2], x1[3]));
                    }
                }
            }
        }
        __syncthreads();                                   // the stage (and red) may be written again
        if (++stage == STAGES) stage = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!p.want_params) return;
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.C;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int c = 2 * (k0 + j * 64);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float vg = lane_sum(ag[j][e], 8), vb = lane_sum(ab[j][e], 8);
            if (l == 0 && c < p.C) {
                out[c + e] = vg;
                out[p.C + c + e] = vb;
            }
        }
    }
}

constexpr int kSmemMost = 200 * 1024;
constexpr int kBlocksPerSm = 2;       // backward grid, in blocks per SM

int chunk_of(int C, int tiles_held, int other_bytes) {
    const int64_t most = (kSmemMost - other_bytes) / (tiles_held * kPitch * 4);
    if (C <= most) return C;
    return (int)(most / 32 * 32);
}

template <typename T, int PP>
cudaError_t fwd_planes(PlaneParams p, cudaStream_t st) {
    p.tiles = (p.rows + kWords * PP - 1) / (kWords * PP);
    p.chunk = chunk_of(p.C, 1, 0);
    const int smem = p.chunk * kPitch * 4;
    cudaError_t e = cudaFuncSetAttribute(planes_fwd_kernel<T, PP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)device_sm_count() * 8;
    if (grid > p.tiles) grid = p.tiles;
    return launch_after(planes_fwd_kernel<T, PP>, dim3((unsigned)grid), dim3(kFwdThreads), smem, st, p);
}

template <typename T, int PP>
cudaError_t bwd_planes(PlaneParams p, int* parts, cudaStream_t st) {
    p.tiles = (p.rows + kWords * PP - 1) / (kWords * PP);
    p.chunk = chunk_of(p.C, 2, 3 * p.C * 4);
    const int smem = 2 * p.chunk * kPitch * 4 + 3 * p.C * 4;
    cudaError_t e = cudaFuncSetAttribute(planes_bwd_kernel<T, PP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)device_sm_count() * kBlocksPerSm;
    if (grid > p.tiles) grid = p.tiles;
    *parts = (int)grid;
    return launch_after(planes_bwd_kernel<T, PP>, dim3((unsigned)grid), dim3(kBwdThreads), smem, st, p);
}

// Whether the 16-bit form serves the call: a plane is whole groups of four
// pixels, rows whole 16-byte vectors, and a thread holds all of its channels.
bool fast16(const layernorm_desc& d, const void* x, const void* dx, const void* rows) {
    return d.dtype != CONV2D_F32 && d.pixels % 4 == 0 && d.cols % 8 == 0 && d.cols <= 1024 && d.ys % 8 == 0 &&
           aligned_to(x, 8) && aligned_to(dx, 8) && aligned_to(rows, 16);
}

template <typename T> cudaError_t fwd_fast(PlaneParams p, cudaStream_t st) {
    const int64_t tiles = (p.rows + kTile - 1) / kTile;
    const size_t smem = (size_t)kTile * ((p.C + 63) / 64 * 64) * 2;
    const dim3 grid((unsigned)tiles);
    const int pairs = (p.C / 2 + 31) / 32;                 // per thread of 256
    if (pairs <= 1) return launch_after(planes16_fwd_kernel<T, 1, 256>, grid, dim3(256), smem, st, p);
    if (pairs <= 2) return launch_after(planes16_fwd_kernel<T, 2, 256>, grid, dim3(256), smem, st, p);
    if (pairs <= 4) return launch_after(planes16_fwd_kernel<T, 4, 256>, grid, dim3(256), smem, st, p);
    if (pairs <= 8) return launch_after(planes16_fwd_kernel<T, 8, 256>, grid, dim3(256), smem, st, p);
    const cudaError_t e = cudaFuncSetAttribute(planes16_fwd_kernel<T, 8, 512>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(planes16_fwd_kernel<T, 8, 512>, grid, dim3(512), smem, st, p);
}

template <typename T, int NP> cudaError_t bwd_fast_np(PlaneParams p, int* parts, cudaStream_t st) {
    p.tiles = (p.rows + kTile - 1) / kTile;
    const size_t stage = (size_t)NP * 8192 + (size_t)kTile * ((p.C + 63) / 64 * 64) * 2;
    const size_t smem = (NP == 8 ? 1 : 3) * stage + (size_t)p.C * 4;
    const cudaError_t e = cudaFuncSetAttribute(planes16_bwd_kernel<T, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (int64_t)device_sm_count() * (NP <= 2 ? 2 : 1);
    if (grid > p.tiles) grid = p.tiles;
    *parts = (int)grid;
    return launch_after(planes16_bwd_kernel<T, NP>, dim3((unsigned)grid), dim3(512), smem, st, p);
}

template <typename T> cudaError_t bwd_fast(const PlaneParams& p, int* parts, cudaStream_t st) {
    const int pairs = (p.C / 2 + 63) / 64;                 // per thread of 512
    if (pairs <= 1) return bwd_fast_np<T, 1>(p, parts, st);
    if (pairs <= 2) return bwd_fast_np<T, 2>(p, parts, st);
    if (pairs <= 4) return bwd_fast_np<T, 4>(p, parts, st);
    return bwd_fast_np<T, 8>(p, parts, st);
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

cudaError_t launch_layernorm_planes_fwd(const layernorm_desc& d, const void* x, const void* gamma, const void* beta,
                                        void* y, float* mean, float* rstd, cudaStream_t st) {
    PlaneParams p = params_of(d);
    p.x = x; p.gamma = gamma; p.beta = beta; p.y = y; p.mean = mean; p.rstd = rstd;
    if (fast16(d, x, nullptr, y))
        return d.dtype == CONV2D_F16 ? fwd_fast<__half>(p, st) : fwd_fast<__nv_bfloat16>(p, st);
    p.pair_c = pair_channels(d, y);
    const bool pair = pair_pixels(d, x, x);
    switch (d.dtype) {
        case CONV2D_F32: return fwd_planes<float, 1>(p, st);
        case CONV2D_F16: return pair ? fwd_planes<__half, 2>(p, st) : fwd_planes<__half, 1>(p, st);
        default: return pair ? fwd_planes<__nv_bfloat16, 2>(p, st) : fwd_planes<__nv_bfloat16, 1>(p, st);
    }
}

size_t layernorm_planes_bwd_workspace(const layernorm_desc& d) {
    return (size_t)device_sm_count() * kBlocksPerSm * 2 * (size_t)d.cols * sizeof(float);
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
        e = d.dtype == CONV2D_F16 ? bwd_fast<__half>(p, &parts, st) : bwd_fast<__nv_bfloat16>(p, &parts, st);
    } else switch (d.dtype) {
        case CONV2D_F32: e = bwd_planes<float, 1>(p, &parts, st); break;
        case CONV2D_F16: e = pair ? bwd_planes<__half, 2>(p, &parts, st) : bwd_planes<__half, 1>(p, &parts, st); break;
        default: e = pair ? bwd_planes<__nv_bfloat16, 2>(p, &parts, st) : bwd_planes<__nv_bfloat16, 1>(p, &parts, st);
    }
    if (e != cudaSuccess || !p.want_params) return e;
    return launch_layernorm_params(p.part, parts, d, dgamma, dbeta, st);
}

}  // namespace conv2d_gb300
