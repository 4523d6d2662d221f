// The feed-forward block's activations and their slopes.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/head.h"

namespace conv2d_gb300 {

// act(g) and its slope.  FAST (16-bit results): approximate exponentials and reciprocals, good to
// 2^-21.  Else the exponential's argument is multiplied by log2 e in two parts, which leaves the approximation's
// 2^-22, and the reciprocal takes a Newton step: a third of the instructions of expf and a division, which
// a tile's only pass through the epilogue would wait for.
// `more`, below 2^-12, is added to x (!FAST).
template <bool FAST> __device__ __forceinline__ float exp_of(float x, float more = 0.f) {
    if constexpr (FAST) return __expf(x);
    constexpr float hi = 1.4426950216293335f, lo = 1.9259629911e-8f, ln2 = 0.69314718055994531f;
    const float t = x * hi, rest = fmaf(x, lo, fmaf(x, hi, -t));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return t > -127.f ? fmaf(e, fmaf(rest, ln2, more), e) : 0.f;       // (`rest` of an infinity is none)
}
template <bool FAST> __device__ __forceinline__ float inverse_of(float x) {      // x in [1, 8]
    if constexpr (FAST) return __fdividef(1.f, x);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return fmaf(r, fmaf(-x, r, 1.f), r);
}
// 1 / (1 + exp(-z)) and what it is from 1, neither by a difference.
template <bool FAST> __device__ __forceinline__ void sigmoid(float z, float& s, float& q) {
    const float e = exp_of<FAST>(-fabsf(z)), r = inverse_of<FAST>(1.f + e), er = e * r;
    s = z >= 0.f ? r : er;
    q = z >= 0.f ? er : r;
    if (isnan(z)) s = q = z;
}
template <int ACT, bool FAST> __device__ __forceinline__ void activate(float g, float& a, float& slope) {
    if constexpr (ACT == FFN_SILU) {
        float s, q;
        sigmoid<FAST>(g, s, q);
        a = g * s;
        slope = s * fmaf(g, q, 1.f);
    } else if constexpr (ACT == FFN_GELU) {
        float phi, e;
        if constexpr (FAST) {
            e = exp_of<true>(-0.5f * g * g);
            // The tail 1 - Phi(|g|) by a polynomial in 1 / (1 + p x) times exp(-x^2), x = |g| / sqrt 2 (the form of
            // Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, with a term more and coefficients
            // fitted to both ends): off by 1.5e-7 at most, and by 2^-15 of itself, which is less than the result's rounding
            // takes.  The slope wants that exponential too, and erff takes three times as long.
            const float t = inverse_of<true>(fmaf(0.29698485f, fabsf(g), 1.f));
            float q = fmaf(t, -0.163697064f, 0.477346015f);
            q = fmaf(t, q, -0.0802607116f);
            q = fmaf(t, q, 0.307915881f);
            q = fmaf(t, q, 0.220616f);
            q = fmaf(t, q, 0.238079579f);
            q *= 0.5f * t * e;
            phi = g > 0.f ? 1.f - q : q;
            if (isnan(g)) phi = g;
        } else {
            // Half of 1 + erff(g / sqrt 2) would cancel below zero (4 % of it is lost at -5), so the tail comes from a
            // polynomial here too, fitted for the least relative error over [0, 14.5]: 2^-26, and 2^-21 with its own
            // roundings.  The square's rounding goes into the exponent.  (Past 20 the exponential is zero.)
            const float gg = g * g, t = inverse_of<false>(fmaf(0.26516503f, fminf(fabsf(g), 20.f), 1.f));
            e = exp_of<false>(-0.5f * gg, -0.5f * fmaf(g, g, -gg));
            float q = fmaf(t, 0.06125977f, -0.286015247f);
            q = fmaf(t, q, 0.429762213f);
            q = fmaf(t, q, -0.226484068f);
            q = fmaf(t, q, 0.271756406f);
            q = fmaf(t, q, 0.122322229f);
            q = fmaf(t, q, 0.205109086f);
            q = fmaf(t, q, 0.210677758f);
            q = fmaf(t, q, 0.211611851f);
            q *= 0.5f * t * e;
            phi = g > 0.f ? 1.f - q : q;
            if (isnan(g)) phi = g;
        }
        a = g * phi;
        slope = fmaf(g * 0.39894228040143268f, e, phi);
    } else {
        // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3).
        constexpr float k = 1.5957691216057308f, c = 0.044715f;      // 2 sqrt(2 / pi)
        float s, q;
        const float gg = g * g;
        sigmoid<FAST>(k * g * fmaf(c, gg, 1.f), s, q);
        a = g * s;
        // (Where s q is zero, the cubic term may have overflowed.)
        const float sq = s * q;
        slope = sq > 0.f ? fmaf(g * k * fmaf(3.f * c, gg, 1.f), sq, s) : s;
    }
}
// act(g) alone, where its slope is not wanted: for silu and gelu_tanh an exponential that may overflow is in its
// place, 1 / (1 + inf) being 0.
template <int ACT, bool FAST> __device__ __forceinline__ float activated(float g) {
    if constexpr (FAST && ACT != FFN_GELU) {
        constexpr float k = 1.5957691216057308f, c = 0.044715f, log2e = 1.4426950408889634f;
        const float z = ACT == FFN_SILU ? -log2e * g : -log2e * k * g * fmaf(c, g * g, 1.f);
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return g * r;
    } else {
        float a, slope;
        activate<ACT, FAST>(g, a, slope);
        return a;
    }
}
// f(a, slope) for each of N pre-activations.
template <bool FAST, int N, typename F> __device__ __forceinline__ void activate_all(int act, const float (&g)[N], F f) {
    const auto each = [&](auto kind) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float a, slope;
            activate<decltype(kind)::value, FAST>(g[j], a, slope);
            f(j, a, slope);
        }
    };
    if (act == FFN_SILU) each(std::integral_constant<int, FFN_SILU>{});
    else if (act == FFN_GELU) each(std::integral_constant<int, FFN_GELU>{});
    else each(std::integral_constant<int, FFN_GELU_TANH>{});
}
// f(a) for each of them.
template <bool FAST, int N, typename F> __device__ __forceinline__ void activated_all(int act, const float (&g)[N], F f) {
    const auto each = [&](auto kind) {
#pragma unroll
        for (int j = 0; j < N; ++j) f(j, activated<decltype(kind)::value, FAST>(g[j]));
    };
    if (act == FFN_SILU) each(std::integral_constant<int, FFN_SILU>{});
    else if (act == FFN_GELU) each(std::integral_constant<int, FFN_GELU>{});
    else each(std::integral_constant<int, FFN_GELU_TANH>{});
}

}  // namespace conv2d_gb300
