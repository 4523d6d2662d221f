// AdamW over many tensors at once, in place, with moments of 32 or 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2   (g times the gradient scale)
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// and, where wanted, a 16-bit copy of p for the products of the next step.  The
// tensors' addresses travel as the kernel's parameter, so a step of up to kMany
// tensors is one launch that needs no workspace and no copy of a table; a block of
// threads finds its tensor by bisection over the tensors' first blocks.
//
// A warp takes 256 adjacent elements, eight a lane: 32-byte loads of fp32 values.
// They are also the blocks of the 8-bit moments (m e4m3, v e5m2): the block's
// largest value, found by one reduction over the warp, fixes a power of two that
// takes it to the type's top binade, and every value goes to one of its two
// neighbours there, up with the chance that keeps the mean.  Rounding to nearest
// would leave a moment where it is forever (b2 = 0.999 moves v by a thousandth a step,
// half a step of e5m2 is a sixteenth); this way it moves as the formula does on
// average.  With the moments in integers of their bits that is one addition of 16
// random bits below the kept ones: Philox4x32-10 under key = seed and counter =
// (element / 4, tensor, step mod 2^32, step div 2^32), one 32-bit word an element, its
// low half for m, its high half for v.  A positive v never becomes zero: m would
// be divided by what a single gradient leaves.  The step itself takes the
// moments before they are rounded.
//
// Where p, g or the copy are not aligned for vectors, and at a tensor's end, a
// warp's elements go through shared memory, so that global memory is read and
// written along the row all the same.
//
// Measured with bf16 gradients and copies, 319 million parameters: fp32 moments 1254 us (7.1 TB/s of 28 bytes a
// parameter; memory bounds it), 8 bits 927 us (5.5 TB/s of 16).  There instructions bound it, 88 a
// parameter of which the generator takes some 15: 1364 us at first; codes without conversions between integers and floats,
// which run at an eighth of the rate, 1172; a warp's next blocks by asynchronous copies, eight blocks a warp, 927 (the
// same by registers 1479: the loop waits for what it moves).
#include <math.h>

#include <type_traits>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kBlock = 256, kLane = 8;                 // elements of a warp and of a lane
// Warps of a block of threads, each with 256 elements at a time; 8 bits: blocks that a warp has on their way or at work.
template <bool EIGHT> __host__ __device__ constexpr int warps() { return EIGHT ? 4 : 8; }
constexpr int kSlots = 3;
template <typename G> __host__ __device__ constexpr int slot_bytes() { return kBlock * (4 + (int)sizeof(G) + 2); }
// Tensors a launch: 1 KB and 31 KB of parameters (the larger ones cost a launch 0.3 to 0.5 us: 5 k parameters 2.9 and 3.2).
constexpr int kFew = 24, kMany = 700;

struct AdamTensor {
    float* p;
    const void* g;
    void* copy;
    int64_t n;
    uint32_t state;          // its first block of 256 in the moments
    float decay;
};

struct AdamStep {
    void *m, *v;
    uint8_t *ms, *vs;        // 8 bits: the blocks' scales (e8m0)
    const int64_t* step_at;  // null: `step`, with the corrections below
    const float* lr_at;      // null: `lr`
    const float* scale;      // null: 1
    const float* skip;       // null, or not zero: nothing changes
    int64_t step;
    float lr, c1, rc2;       // 1 - b1^t, 1 / sqrt(1 - b2^t)
    float log_b1, log_b2;
    float b1, b2, a1, a2, eps;     // a = 1 - b
    uint32_t k0, k1;
    uint32_t first_tensor;   // number of the launch's first tensor
    int copy_bf16, count;
    int span;                // blocks of 256 that a warp takes
};

template <int N> struct AdamTable {
    AdamTensor t[N];
    uint32_t first[N + 1];   // a tensor's first block of threads
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    uint32_t r[8];
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(f[i]);
    st_global_v8(p, r);
}
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
    widen(*reinterpret_cast<const Vec<T, 8>*>(p), f);
}

// Eight values of 8 bits.  An e5m2 code is the high byte of an fp16 value; an e4m3 one,
// its magnitude moved down by a bit, that of 2^-8 times its own, subnormal values
// included.  (Conversions from integers run at an eighth of the rate.)
template <bool E4M3> __device__ __forceinline__ void from8(uint2 c, uint32_t byte, float (&f)[8]) {
    // The scale 2^(byte - 127): 255 is not a number, 2^-127 no normal value (but 2^-119 is).
    const uint32_t b = byte + (E4M3 ? 8u : 0u);
    const float scale = __uint_as_float(byte == 255u ? 0x7fffffffu : b ? b << 23 : 0x00400000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h = __byte_perm(i < 2 ? c.x : c.y, 0u, i & 1 ? 0x3424 : 0x1404);      // each code in a high byte
        if (E4M3) h = (h & 0x80008000u) | (h >> 1 & 0x3f803f80u);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// The same back, DIGITS bits of the significand after the leading one.  `most`: the
// bits of the block's largest magnitude.  r: the elements' numbers, whose low (m) or
// high (v) half is the noise.  Below the lowest normal value, 2^LOW, that value is added: the
// bits then count the steps of the subnormal values (the sum is cut, not rounded).
template <bool E4M3> __device__ __forceinline__ uint2 to8(const float (&f)[8], uint32_t most, const uint32_t (&r)[8],
                                                          uint32_t& byte) {
    constexpr int kDigits = E4M3 ? 3 : 2, kLow = E4M3 ? -6 : -14, kTop = E4M3 ? 8 : 15, kDrop = 23 - kDigits;
    constexpr uint32_t kBase = (uint32_t)(kLow + 126) << kDigits;
    const float least = __uint_as_float((uint32_t)(127 + kLow) << 23);
    // One binade more where the largest is above 1.75 of its own: what rounding up
    // makes of it still fits.
    const int exponent = (int)((most + (1u << 21) - 1u) >> 23) - 127;
    const int scale = max(exponent - kTop, -127);
    byte = most >= 0x7f800000u ? 255u : (uint32_t)(scale + 127);
    const float up = __uint_as_float((uint32_t)(127 - scale) << 23);
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t noise = E4M3 ? (r[i] & 0xffffu) << (kDrop - 16) : r[i] >> 16 << (kDrop - 16);
        const float y = fabsf(f[i]) * up;
        const bool small = y < least;
        const uint32_t bits = __float_as_uint(small ? __fadd_rz(y, least) : y);
        code[i] = (bits + noise - (small ? (kBase << kDrop) + (1u << 23) : kBase << kDrop)) >> kDrop;
        if (E4M3) code[i] |= __float_as_uint(f[i]) >> 24 & 0x80u;
        else code[i] = max(code[i], min(__float_as_uint(f[i]), 1u));      // v: above zero stays above zero, also where y does not
    }
    if (byte == 255u) return make_uint2(0u, 0u);
    const auto four = [&](int i) {
        return __byte_perm(__byte_perm(code[i], code[i + 1], 0x0040), __byte_perm(code[i + 2], code[i + 3], 0x0040), 0x5410);
    };
    return make_uint2(four(0), four(4));
}

// m / (sqrt(v) k + eps), the root and the reciprocal off by 2^-23 each at most, which p sees times lr.  The reciprocal takes
// no subnormal numbers, but eps is 2^-126 at least.  Neither does the faster root: v below 2^-126 counts as that
// there (and one that is not a number as it is), which takes part only where 2^-63 k is 2^-26 of eps at most.  (8 bits, 256 M
// parameters: 777 us with that one, 796 with the other for all.)
template <bool SUBNORMAL> __device__ __forceinline__ float update(float m, float v, float k, float eps) {
    float root, inverse;
    if constexpr (SUBNORMAL) {
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
    } else {
        float normal;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(normal) : "f"(v), "f"(0x1p-126f));
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(normal));
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inverse) : "f"(fmaf(root, k, eps)));
    return m * inverse;
}

template <typename G, bool EIGHT, int N>
__global__ void __launch_bounds__(32 * warps<EIGHT>(), EIGHT ? 7 : 4)
adamw_kernel(const __grid_constant__ AdamTable<N> table, const __grid_constant__ AdamStep s) {
    constexpr int kWarps = warps<EIGHT>();
    // A warp's blocks on their way (8 bits), or one block of a tensor's elements on their way between the lanes.
    __shared__ __align__(16) float stage[kWarps][(EIGHT ? kSlots * slot_bytes<G>() : (kBlock + kBlock / 8) * 4) / 4];
    // The last tensor whose first block is not past this one.
    int lo = 0, hi = s.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const AdamTensor t = table.t[lo];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i0 = lane * kLane;
    // An element's place in the stage: eight in a row, then one to spare.
    float* const row = stage[warp];
    const auto place = [](int e) { return e + (e >> 3); };
    pdl_wait();
    if (s.skip && *s.skip != 0.f) return;
    int64_t step = s.step;
    float c1 = s.c1, rc2 = s.rc2;
    if (s.step_at) {
        step = *s.step_at;
        c1 = -expm1f((float)step * s.log_b1);
        rc2 = 1.f / sqrtf(-expm1f((float)step * s.log_b2));
    }
    const float lr = s.lr_at ? *s.lr_at : s.lr, up = lr / c1, shrink = fmaf(-lr, t.decay, 1.f);
    const float k = s.scale ? *s.scale : 1.f;
    const bool eps_hides = rc2 * 0x1p-37f <= s.eps;        // the root of 2^-126
    int64_t e0 = ((int64_t)(blockIdx.x - table.first[lo]) * s.span * kWarps + warp) * kBlock;
    const bool aligned = (reinterpret_cast<uintptr_t>(t.p) & 31u) == 0 &&
                         (reinterpret_cast<uintptr_t>(t.g) & (sizeof(G) * 8 - 1)) == 0 &&
                         (reinterpret_cast<uintptr_t>(t.copy) & 15u) == 0;
    const auto is_whole = [&](int64_t e) { return aligned && e + kBlock <= t.n; };
    // In 8 bits a warp has more arithmetic than its own loads can hide: the next two whole blocks are on their way
    // to shared memory meanwhile, every lane's own values in its own places.
    constexpr uint32_t kG = kBlock * 4, kM = kG + kBlock * sizeof(G), kV = kM + kBlock;      // p, g, m, v in a slot
    const auto slot = [&](int j) { return reinterpret_cast<uint8_t*>(row) + j % kSlots * slot_bytes<G>(); };
    const auto fetch = [&](int j) {
        const int64_t e = e0 + (int64_t)j * kWarps * kBlock;
        if (j < s.span && is_whole(e)) {
            const uint32_t to = smem_addr(slot(j)) + 16 * lane;
            const int64_t at = (int64_t)t.state * kBlock + e;
#pragma unroll
            for (int h = 0; h < 2; ++h) copy_async<16>(to + 512 * h, t.p + e + i0 + 4 * h);
#pragma unroll
            for (int h = 0; h < (int)sizeof(G) / 2; ++h)
                copy_async<16>(to + kG + 512 * h, static_cast<const G*>(t.g) + e + i0 + 4 * h);
            copy_async<8>(to + kM - 8 * lane, static_cast<const uint8_t*>(s.m) + at + i0);
            copy_async<8>(to + kV - 8 * lane, static_cast<const uint8_t*>(s.v) + at + i0);
        }
        copy_async_commit();
    };
    uint32_t scales_m = 0, scales_v = 0;                   // lane j's: those of the warp's block j
    if constexpr (EIGHT) {
        fetch(0);
        fetch(1);
        const int64_t at = (int64_t)t.state + e0 / kBlock + lane * kWarps;
        if (lane < s.span && e0 + (int64_t)lane * kWarps * kBlock < t.n) {
            scales_m = s.ms[at];
            scales_v = s.vs[at];
        }
    }
    const int64_t first = e0;
#pragma unroll 1
    for (int j = 0; j < (EIGHT ? s.span : 1); ++j) {
        const int64_t e0 = first + (int64_t)j * kWarps * kBlock;
        if (e0 >= t.n) break;
        const int64_t at = (int64_t)t.state * kBlock + e0;     // in the moments
        const int left = (int)min((int64_t)kBlock, t.n - e0);
        float* p = t.p + e0;
        const G* g = static_cast<const G*>(t.g) + e0;
        uint16_t* copy = t.copy ? static_cast<uint16_t*>(t.copy) + e0 : nullptr;
        const bool whole = is_whole(e0);
        float fp[8], fg[8], fm[8], fv[8];
        uint32_t bm = 0, bv = 0;
        if constexpr (EIGHT) {
            bm = __shfl_sync(0xffffffffu, scales_m, j);
            bv = __shfl_sync(0xffffffffu, scales_v, j);
            uint2 cm, cv;
            if (whole) {
                copy_async_wait<1>();
                const uint8_t* at = slot(j);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    widen(reinterpret_cast<const Vec<float, 4>*>(at + 512 * h)[lane],
                          *reinterpret_cast<float(*)[4]>(fp + 4 * h));
                if constexpr (sizeof(G) == 4) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        widen(reinterpret_cast<const Vec<float, 4>*>(at + kG + 512 * h)[lane],
                              *reinterpret_cast<float(*)[4]>(fg + 4 * h));
                } else {
                    widen(reinterpret_cast<const Vec<G, 8>*>(at + kG)[lane], fg);
                }
                cm = reinterpret_cast<const uint2*>(at + kM)[lane];
                cv = reinterpret_cast<const uint2*>(at + kV)[lane];
                fetch(j + 2);                              // (where block j - 1 was)
            } else {
                cm = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.m) + at)[lane];
                cv = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.v) + at)[lane];
            }
            from8<true>(cm, bm, fm);
            from8<false>(cv, bv, fv);
        } else {
            if (whole) {
                load8(p + i0, fp);
                load8(g + i0, fg);
            }
            load8(static_cast<const float*>(s.m) + at + i0, fm);
            load8(static_cast<const float*>(s.v) + at + i0, fv);
        }
        const uint32_t nan_m = EIGHT && bm == 255u ? 0x7fffffffu : 0u;
        if (!whole) {
            __syncwarp();
            for (int e = lane; e < kBlock; e += 32) row[place(e)] = e < left ? p[e] : 0.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) fp[i] = row[place(i0 + i)];
            __syncwarp();
            for (int e = lane; e < kBlock; e += 32) row[place(e)] = e < left ? to_f32(g[e]) : 0.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) fg[i] = row[place(i0 + i)];
        }
        if (s.scale) {
#pragma unroll
            for (int i = 0; i < 8; ++i) fg[i] *= k;
        }
        if (!whole) {                                          // past the end: zero, whatever lies there
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i >= left) fm[i] = fv[i] = 0.f;
        }
        float top_m = 0.f;
        uint32_t top_v = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // Each product and sum rounds by itself: the 8-bit codes are then a matter of the formula alone, not of which of
            // them a compiler joins.
            fm[i] = __fadd_rn(__fmul_rn(s.b1, fm[i]), __fmul_rn(s.a1, fg[i]));
            fv[i] = __fadd_rn(__fmul_rn(s.b2, fv[i]), __fmul_rn(__fmul_rn(s.a2, fg[i]), fg[i]));
            top_m = fmaxf(top_m, fabsf(fm[i]));
            top_v = max(top_v, __float_as_uint(fv[i]));
        }
        const auto step_all = [&](auto subnormal) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                fp[i] = fmaf(-up, update<decltype(subnormal)::value>(fm[i], fv[i], rc2, s.eps), fp[i] * shrink);
        };
        if (eps_hides) step_all(std::false_type{});
        else step_all(std::true_type{});
        if (whole) {
            store8(p + i0, fp);
            if (copy) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x2 two = pack2f(fp[2 * i], fp[2 * i + 1]);
                    w[i] = s.copy_bf16 ? narrow_pair<__nv_bfloat16>(two) : narrow_pair<__half>(two);
                }
                *reinterpret_cast<uint4*>(copy + i0) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) row[place(i0 + i)] = fp[i];
            __syncwarp();
            for (int e = lane; e < left; e += 32) {
                const float f = row[place(e)];
                p[e] = f;
                if (copy) store_param(copy, false, s.copy_bf16, e, f);
            }
        }
        if constexpr (EIGHT) {
            uint32_t r[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t c[4] = {(uint32_t)(e0 / 4) + 2 * lane + k, s.first_tensor + lo, (uint32_t)step,
                                 (uint32_t)((uint64_t)step >> 32)};
                philox(c, s.k0, s.k1);
#pragma unroll
                for (int i = 0; i < 4; ++i) r[4 * k + i] = c[i];
            }
            // A NaN, which the maximum of floats passes over, is in m only where it was, or where one in g makes v's.
            top_v = __reduce_max_sync(0xffffffffu, top_v);
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top_m));
            const uint2 cm = to8<true>(fm, top_v > 0x7f800000u ? top_v : max(most, nan_m), r, bm);
            const uint2 cv = to8<false>(fv, top_v, r, bv);
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.m) + at)[lane] = cm;
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.v) + at)[lane] = cv;
            if (lane == 0) {
                s.ms[at / kBlock] = (uint8_t)bm;
                s.vs[at / kBlock] = (uint8_t)bv;
            }
        } else {
            store8(static_cast<float*>(s.m) + at + i0, fm);
            store8(static_cast<float*>(s.v) + at + i0, fv);
        }
    }
}

// Blocks of 256 that a warp takes one after the other (at most 32: a lane keeps the scales of one).  In 8 bits eight
// keep the copies going where there are enough of them for the machine: one / eight, 1 M parameters 6.3 / 9.3 us, 4 M 17.3 /
// 20.0, 16 M 59.5 / 56.8, 64 M 226 / 201, 256 M 892 / 777.
int span_of(const adamw_desc& d) { return d.states == ADAMW_STATES_8BIT && d.elements >= (1 << 24) ? 8 : 1; }

// Blocks of threads for n elements.
int64_t blocks_of(int64_t n, bool eight, int span) {
    const int64_t each = (int64_t)kBlock * (eight ? warps<true>() : warps<false>()) * span;
    return (n + each - 1) / each;
}

template <typename G, bool EIGHT, int N>
cudaError_t launch(const adamw_desc& d, int from, int count, float* const* params, const void* const* grads,
                   void* const* copies, AdamStep s, int span, cudaStream_t st) {
    AdamTable<N> table;
    uint32_t blocks = 0;
    s.span = span;
    int k = 0;
    for (int i = from; i < from + count; ++i) {
        // (An empty tensor keeps its number and takes no block.)
        table.t[k] = AdamTensor{params[i], grads[i], copies ? copies[i] : nullptr, d.tensors[i].n,
                                (uint32_t)(d.tensors[i].offset / kBlock), d.tensors[i].decay};
        table.first[k++] = blocks;
        blocks += (uint32_t)blocks_of(d.tensors[i].n, EIGHT, span);
    }
    if (!blocks) return cudaSuccess;
    s.first_tensor = (uint32_t)from;
    s.count = count;
    return launch_after(adamw_kernel<G, EIGHT, N>, dim3(blocks), dim3(32 * warps<EIGHT>()), 0, st, table, s);
}

template <typename G, bool EIGHT>
cudaError_t run(const adamw_desc& d, float* const* params, const void* const* grads, void* const* copies,
                const AdamStep& s, cudaStream_t st) {
    const int count = d.count, span = span_of(d);
    for (int from = 0; from < count;) {
        // As many tensors as a launch's table and its number of blocks take.
        int n = 0;
        int64_t blocks = 0;
        while (from + n < count && n < kMany) {
            const int64_t more = blocks_of(d.tensors[from + n].n, EIGHT, span);
            if (n && blocks + more > 0x7fffffffLL) break;
            blocks += more;
            ++n;
        }
        const cudaError_t e = n <= kFew ? launch<G, EIGHT, kFew>(d, from, n, params, grads, copies, s, span, st)
                                        : launch<G, EIGHT, kMany>(d, from, n, params, grads, copies, s, span, st);
        if (e != cudaSuccess) return e;
        from += n;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const adamw_desc& d, float* const* params, const void* const* grads, void* const* copies,
                         void* m, void* v, void* m_scale, void* v_scale, int64_t step, float lr,
                         const int64_t* step_at, const float* lr_at, const float* grad_scale, const float* skip,
                         uint64_t seed, cudaStream_t st) {
    AdamStep s{};
    s.m = m;
    s.v = v;
    s.ms = static_cast<uint8_t*>(m_scale);
    s.vs = static_cast<uint8_t*>(v_scale);
    s.step_at = step_at;
    s.lr_at = lr_at;
    s.scale = grad_scale;
    s.skip = skip;
    s.step = step;
    s.lr = lr;
    if (!step_at) {
        s.c1 = (float)(1.0 - pow(d.beta1, (double)step));
        s.rc2 = (float)(1.0 / sqrt(1.0 - pow(d.beta2, (double)step)));
    }
    s.log_b1 = (float)log(d.beta1);
    s.log_b2 = (float)log(d.beta2);
    s.b1 = (float)d.beta1; s.a1 = (float)(1.0 - d.beta1);
    s.b2 = (float)d.beta2; s.a2 = (float)(1.0 - d.beta2);
    s.eps = (float)d.eps;
    s.k0 = (uint32_t)seed;
    s.k1 = (uint32_t)(seed >> 32);
    s.copy_bf16 = d.copy == CONV2D_BF16;
    const bool eight = d.states == ADAMW_STATES_8BIT;
    switch (d.grad) {
        case CONV2D_F32:
            return eight ? run<float, true>(d, params, grads, copies, s, st)
                         : run<float, false>(d, params, grads, copies, s, st);
        case CONV2D_F16:
            return eight ? run<__half, true>(d, params, grads, copies, s, st)
                         : run<__half, false>(d, params, grads, copies, s, st);
        default:
            return eight ? run<__nv_bfloat16, true>(d, params, grads, copies, s, st)
                         : run<__nv_bfloat16, false>(d, params, grads, copies, s, st);
    }
}

}  // namespace conv2d_gb300
