// Element types and 16-byte vectors of the training-head kernels: values are
// widened to fp32 on load and rounded to nearest even once on store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace conv2d_gb300 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V adjacent elements as they lie in memory; aligned so that a full 16-byte
// vector is one load.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

template <typename T, int V> __device__ __forceinline__ void widen(const Vec<T, V>& a, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(a.v[i]);
}
template <typename T, int V> __device__ __forceinline__ Vec<T, V> narrow(const float (&f)[V]) {
    Vec<T, V> a;
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = from_f32<T>(f[i]);
    return a;
}

// Elements [lo, hi) of a vector whose first element is p[0]: one load when it
// is whole, else one by one with zeros outside (nothing outside is read).
template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_part(const T* p, int lo, int hi) {
    Vec<T, V> a;
    if (lo == 0 && hi == V) {
        a = *reinterpret_cast<const Vec<T, V>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) a.v[i] = i >= lo && i < hi ? p[i] : from_f32<T>(0.f);
    }
    return a;
}
template <typename T, int V> __device__ __forceinline__ void store_part(T* p, const Vec<T, V>& a, int lo, int hi) {
    if (lo == 0 && hi == V) {
        *reinterpret_cast<Vec<T, V>*>(p) = a;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= lo && i < hi) p[i] = a.v[i];
    }
}

// Elements [lo, hi) of the V parameters from column e0 on, of type T or fp32
// (`f32`); `fill` outside, and everywhere when there are none (null).  `vec`
// says that a whole vector may be read with 16-byte loads.  Parameters are read
// as constant data: no store of the kernel holds the loads of the next vector back.
template <typename T, int V>
__device__ __forceinline__ void load_params(const void* p, bool f32, int64_t e0, int lo, int hi, bool vec, float fill,
                                            float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = fill;
    if (!p) return;
    const bool whole = vec && V > 1 && lo == 0 && hi == V;
    if (f32) {
        const float* q = static_cast<const float*>(p) + e0;
        if (whole) {
            if constexpr (V >= 4) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 t = __ldg(reinterpret_cast<const float4*>(q + i));
                    f[i] = t.x; f[i + 1] = t.y; f[i + 2] = t.z; f[i + 3] = t.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= lo && i < hi) f[i] = __ldg(q + i);
        }
    } else {
        const T* q = static_cast<const T*>(p) + e0;
        if (whole) {
            if constexpr (V > 1) {
                const uint4 t = __ldg(reinterpret_cast<const uint4*>(q));
                widen<T, V>(*reinterpret_cast<const Vec<T, V>*>(&t), f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= lo && i < hi) f[i] = to_f32(q[i]);
        }
    }
}

__device__ __forceinline__ void store_param(void* p, bool f32, bool bf16, int64_t i, float v) {
    if (f32) static_cast<float*>(p)[i] = v;
    else if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Two fp32 values in a 64-bit register pair: one instruction does both (the
// packed fp32 arithmetic of sm_100 and later; each half rounds as usual).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2f(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pack2f(a, a); }
__device__ __forceinline__ void unpack2f(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum_halves(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    return a + b;
}

// A packed pair of 16-bit values to and from a pair of fp32 ones.
template <typename T> __device__ __forceinline__ f32x2 widen_pair(uint32_t w);
template <> __device__ __forceinline__ f32x2 widen_pair<__nv_bfloat16>(uint32_t w) {
    return pack2f(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ f32x2 widen_pair<__half>(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack2f(f.x, f.y);
}
template <typename T> __device__ __forceinline__ uint32_t narrow_pair(f32x2 v);
template <> __device__ __forceinline__ uint32_t narrow_pair<__nv_bfloat16>(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t narrow_pair<__half>(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A 16-byte vector as pairs of fp32 values, and back.
template <typename T> struct Pairs {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(const uint4& w, f32x2 (&f)[4]) {
        f[0] = widen_pair<T>(w.x); f[1] = widen_pair<T>(w.y); f[2] = widen_pair<T>(w.z); f[3] = widen_pair<T>(w.w);
    }
    static __device__ __forceinline__ uint4 narrow(const f32x2 (&f)[4]) {
        return make_uint4(narrow_pair<T>(f[0]), narrow_pair<T>(f[1]), narrow_pair<T>(f[2]), narrow_pair<T>(f[3]));
    }
};
template <> struct Pairs<float> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void widen(const uint4& w, f32x2 (&f)[2]) {
        f[0] = pack2f(__uint_as_float(w.x), __uint_as_float(w.y));
        f[1] = pack2f(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 narrow(const f32x2 (&f)[2]) {
        float a, b, c, d;
        unpack2f(f[0], a, b);
        unpack2f(f[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
};

// Sum over aligned groups of `width` lanes (a power of two), in every lane.
__device__ __forceinline__ float lane_sum(float v, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// N sums (a power of two) over a warp at once: each exchange also halves the
// values that a lane carries, until lanes k 32 / N on hold sum k.
template <int N> __device__ __forceinline__ float warp_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = N / 2; n > 0; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < n; ++k)
            v[k] = (up ? v[k + n] : v[k]) + __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + n], o);
    }
#pragma unroll
    for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return v[0];
}

// Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011):
// ten rounds of two 32x32-bit products.
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

}  // namespace conv2d_gb300
