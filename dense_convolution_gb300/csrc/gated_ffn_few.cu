// The feed-forward block of few tokens (serving), forward, on the CUDA cores: one pass
// over the three weights is all there is, so they are read in place, whatever their
// type, row length or alignment, and nothing is rounded below fp32 on the way.
//
//   ffn_few_kernel<GATE>   a team of warps takes two rows of Wg and the same two of Wu at
//              a time, each warp a share of their columns, a vector a lane; the
//              tokens' values lie in shared memory (head_few.cuh).  The warps'
//              sums of up to eight such quadruples wait in shared memory; then
//              they are added and h goes out in fp32.
//   ffn_few_kernel<!GATE>  the same over four rows of Wd, with h in shared memory.
//
// The rows of a quadruple are a vector length apart, so that they are offset alike
// against the 16-byte boundary.
//
// Reading the weights bounds it, and two launches of about 4.5 us each that wait for one another: one token, bf16
// 2048 x 8192 25 us (4.0 TB/s), fp16 4096 x 16384 70 us (5.8), fp32 2048 x 8192 41 us (4.9), 512 x 1408 9 us.  Sums that met
// after every quadruple cost 10 % more; fetching the second kernel's rows to the L2 before its wait brought
// nothing, since the first one's blocks fill the machine until then.
#include <type_traits>

#include "gated_ffn_device.cuh"
#include "head_device.cuh"
#include "head_few.cuh"
#include "head_parts.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kRounds = 8;               // quadruples of a team between meetings
constexpr int kSmemMost = 200 * 1024;

struct FfnFew {
    int tokens, cols, rows;      // cols: of the rows that are read; rows: inner, or hidden
    int team;                    // warps
    int token0;                  // first token's number
    int act;
    int64_t xs, ys;              // tokens' row strides, in and out (GATE: out is h, `rows` wide)
    const void *x;               // tokens' values: the operands' type (GATE), or h
    const void *w, *w2;          // Wg and Wu, or Wd
    const void* res;
    float *h, *saved;
    uint16_t* kept;              // h as it is saved
    int64_t fp;                  // saved's columns of g
    void* y;
};

template <typename T, int NT, bool GATE>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) ffn_few_kernel(const FfnFew p) {
    constexpr int V = kVec<T>, kRows = 4, N = kRows * NT, kSpan = 32 / N;
    constexpr int P = kPair<NT>, NP = NT / P, kStep = GATE ? 2 : 4;          // rows of one matrix
    using W = typename Word<P>::T;
    extern __shared__ __align__(16) float hs[];            // [NP][V][pitch][P]
    const W* words = reinterpret_cast<const W*>(hs);
    __shared__ float red[kRounds][kWarps][N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pitch = few_pitch<T>(p.cols), team = warp / p.team, part = warp - team * p.team;
    const int teams = gridDim.x * (kWarps / p.team);
    // Quadruples: a block of kStep V rows and an offset in it below V.
    const int quads = (int)(((int64_t)p.rows + kStep * V - 1) / (kStep * V)) * V;
    const auto row_of = [&](int q) { return q / V * (kStep * V) + q % V; };
    const auto row_at = [&](int r0, int r) {               // row r of the quadruple, and whether it is there
        const T* w = static_cast<const T*>(GATE && r >= 2 ? p.w2 : p.w);
        return w + (int64_t)(r0 + r % kStep * V) * p.cols;
    };
    for (int i = threadIdx.x; i < NT * V * pitch; i += kThreads) hs[i] = 0.f;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    for (int t = 0; t < p.tokens; ++t) {
        for (int e = threadIdx.x; e < p.cols; e += kThreads) {
            const float v = GATE ? to_f32(static_cast<const T*>(p.x)[t * p.xs + e]) : static_cast<const float*>(p.x)[t * p.xs + e];
            hs[((t / P * V + (e & (V - 1))) * pitch + (e >> shift_bits<T>()) + 1) * P + t % P] = v;
        }
    }
    __syncthreads();

    // Rounds of quadruples, as many as their sums have room for; then the teams' sums are added and go out.
    for (int q0 = blockIdx.x * (kWarps / p.team); q0 < quads; q0 += kRounds * teams) {
#pragma unroll 1
        for (int round = 0; round < kRounds; ++round) {
            const int q = q0 + team + round * teams, r0 = row_of(q);
            // (A block's last offsets may have no row at all.)
            if (q >= quads || r0 >= p.rows) continue;
            W acc[kRows][NP];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int t = 0; t < NP; ++t) acc[r][t] = spread<P>(0.f);
            // Wg's rows and Wu's may be offset unlike each other.
            constexpr int kSets = GATE ? 2 : 1, kPer = kRows / kSets;
            const T* base[kSets];
            int shift[kSets], off[kSets][V];
#pragma unroll
            for (int k = 0; k < kSets; ++k) {
                base[k] = row_at(r0, k * kPer);
                shift[k] = phase_of(base[k]);
                word_offsets<T>(shift[k], pitch, off[k]);
            }
            // This warp's share of the slots; whole vectors of four whole rows without tests.
            const int most = max(shift[0], shift[kSets - 1]), slots = (p.cols + most + V - 1) >> shift_bits<T>();
            const int lo = slots * part / p.team, hi = slots * (part + 1) / p.team;
            const bool four = r0 + (kStep - 1) * V < p.rows;
            const int wlo = four ? max(lo, (int)(most != 0)) : hi;
            const int whi = four ? min(hi, (p.cols + min(shift[0], shift[kSets - 1])) >> shift_bits<T>()) : hi;
            const auto run = [&](auto alike) {             // alike: all rows take the same words
                const auto add = [&](const Vec<T, V>(&raw)[kRows], int s) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        W f[kRows];
#pragma unroll
                        for (int r = 0; r < kRows; ++r) f[r] = spread<P>(to_f32(raw[r].v[i]));
#pragma unroll
                        for (int t = 0; t < NP; ++t) {
                            W x = words[t * V * pitch + off[0][i] + s];
#pragma unroll
                            for (int r = 0; r < kRows; ++r) {
                                if (!decltype(alike)::value && r == kPer) x = words[t * V * pitch + off[kSets - 1][i] + s];
                                acc[r][t] = fma_words(f[r], x, acc[r][t]);
                            }
                        }
                    }
                };
#pragma unroll(NT >= 8 ? 1 : 2)
                for (int s = wlo + lane; s < whi; s += 32) {
                    Vec<T, V> raw[kRows];
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        raw[r] = *reinterpret_cast<const Vec<T, V>*>(base[r / kPer] + (int64_t)(r % kPer) * V * p.cols +
                                                                     (s * V - shift[r / kPer]));
                    add(raw, s);
                }
                // The rows' ends, or all slots of rows at the matrix' end.
                for (int j = lo + lane; j < hi; j += 32) {
                    const int s = j < wlo ? j : j + max(0, whi - wlo);
                    if (s >= hi) break;
                    Vec<T, V> raw[kRows];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const bool in = r0 + r % kStep * V < p.rows;
                        const int e0 = s * V - shift[r / kPer];
                        const int from = max(0, -e0), to = max(from, min(V, p.cols - e0));
                        raw[r] = load_part<T, V>(base[r / kPer] + (in ? (int64_t)(r % kPer) * V * p.cols + e0 : 0), in ? from : V,
                                                 in ? to : 0);
                    }
                    add(raw, s);
                }
            };
            if (shift[0] == shift[kSets - 1]) run(std::true_type{});
            else run(std::false_type{});
            float sums[N];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int t = 0; t < NP; ++t) {
                    if constexpr (P == 2) unpack2f(acc[r][t], sums[r * NT + 2 * t], sums[r * NT + 2 * t + 1]);
                    else sums[r] = acc[r][t];
                }
            __syncwarp();
            const float z = warp_sums<N>(sums);
            if (lane % kSpan == 0) red[round][warp][lane / kSpan] = z;
        }
        __syncthreads();
        // A result a thread: of round, team, row and token.
        constexpr int kOut = GATE ? 2 * NT : N;
        for (int i = threadIdx.x; i < kRounds * (kWarps / p.team) * kOut; i += kThreads) {
            const int k = i % kOut, of = i / kOut % (kWarps / p.team), round = i / (kOut * (kWarps / p.team));
            const int q = q0 + of + round * teams, r0 = row_of(q), row = r0 + k / NT * V, t = k % NT;
            if (q >= quads || row >= p.rows || t >= p.tokens) continue;
            const auto total = [&](int k) {
                float f = 0.f;
                for (int j = 0; j < p.team; ++j) f += red[round][of * p.team + j][k];
                return f;
            };
            if constexpr (GATE) {
                const float g = total(k), u = total(k + 2 * NT);
                float h = 0.f;
                const float one[1] = {g};
                activated_all<false>(p.act, one, [&](int, float a) { h = a * u; });
                p.h[(int64_t)t * p.ys + row] = h;
                if (p.saved) {
                    // (As gated_ffn.cu lays it out: up to 32 tokens are one block of rows.)
                    float* at = p.saved + (row / 4) * 128 + (p.token0 + t) * 4 + row % 4;
                    at[0] = g;
                    at[p.fp * 32] = u;
                    uint16_t* kept = p.kept + (int64_t)(p.token0 + t) * p.fp * (sizeof(T) == 4 ? 3 : 1) + row;
                    if constexpr (sizeof(T) == 4) {
                        float part[3];
                        split3(h, part);
#pragma unroll
                        for (int j = 0; j < 3; ++j) reinterpret_cast<__nv_bfloat16*>(kept)[j * p.fp] = __float2bfloat16_rn(part[j]);
                    } else {
                        *reinterpret_cast<T*>(kept) = from_f32<T>(h);
                    }
                }
            } else {
                float y = total(k);
                if (p.res) y += to_f32(static_cast<const T*>(p.res)[(int64_t)t * p.ys + row]);
                static_cast<T*>(p.y)[(int64_t)t * p.ys + row] = from_f32<T>(y);
            }
        }
        __syncthreads();
    }
}

int nt_of(int64_t tokens) { return tokens <= 1 ? 1 : tokens <= 2 ? 2 : tokens <= 4 ? 4 : 8; }

template <typename T> size_t few_smem(int nt, int64_t cols) {
    return (size_t)nt * kVec<T> * few_pitch<T>((int)cols) * sizeof(float);
}

// Warps of a team: few rounds of quadruples, each a lane's vectors of a row and half as long again as one
// for the sums.
int team_of(int cols, int rows, int vec, int step, int blocks) {
    const int quads = (rows + step * vec - 1) / (step * vec) * vec, vectors = (cols + 32 * vec - 1) / (32 * vec);
    int best = 1;
    double least = -1;
    for (int team = 1; team <= kWarps; team *= 2) {
        const int teams = blocks * (kWarps / team);
        const double cost = (double)((quads + teams - 1) / teams) * ((vectors + team - 1) / team + 0.5);
        if (least < 0 || cost < least) {
            least = cost;
            best = team;
        }
    }
    return best;
}

template <typename T, int NT, bool GATE> cudaError_t few_launch(FfnFew p, int sms, cudaStream_t st) {
    const cudaError_t e = allow_smem(ffn_few_kernel<T, NT, GATE>, kSmemMost);
    if (e != cudaSuccess) return e;
    const size_t smem = few_smem<T>(NT, p.cols);
    const int blocks = sms * (NT <= 2 && smem <= 100 * 1024 ? 2 : 1);
    p.team = team_of(p.cols, p.rows, kVec<T>, GATE ? 2 : 4, blocks);
    return launch_after(ffn_few_kernel<T, NT, GATE>, dim3((unsigned)blocks), dim3(kThreads), smem, st, p);
}
template <typename T, bool GATE> cudaError_t few_tokens(const FfnFew& p, int sms, cudaStream_t st) {
    switch (nt_of(p.tokens)) {
        case 1: return few_launch<T, 1, GATE>(p, sms, st);
        case 2: return few_launch<T, 2, GATE>(p, sms, st);
        case 4: return few_launch<T, 4, GATE>(p, sms, st);
        default: return few_launch<T, 8, GATE>(p, sms, st);
    }
}

// Tokens that go through together: up to eight, as many as fit a block's shared memory (0: not even one).
int group_of(const gated_ffn_desc& d) {
    const int64_t cols = d.hidden > d.inner ? d.hidden : d.inner;
    int nt = nt_of(d.tokens);
    while (nt && (d.dtype == CONV2D_F32 ? few_smem<float>(nt, cols) : few_smem<__half>(nt, cols)) > (size_t)kSmemMost) nt /= 2;
    return nt;
}

template <typename T>
cudaError_t run(const gated_ffn_desc& d, const void* x, const void* wg, const void* wu, const void* wd,
                const void* residual, void* y, float* saved, float* h, cudaStream_t st) {
    const int group = group_of(d);
    for (int64_t t = 0; t < d.tokens; t += group) {
        FfnFew p{};
        p.tokens = (int)(d.tokens - t < group ? d.tokens - t : group);
        p.act = d.act;
        p.cols = (int)d.hidden;
        p.rows = (int)d.inner;
        p.xs = d.xs;
        p.ys = d.inner;
        p.x = static_cast<const T*>(x) + t * d.xs;
        p.w = wg;
        p.w2 = wu;
        p.h = h;
        p.fp = (d.inner + 63) / 64 * 64;
        p.saved = saved;
        p.kept = saved ? gated_ffn_saved_h(d, saved) : nullptr;
        p.token0 = (int)t;
        cudaError_t e = few_tokens<T, true>(p, d.sms, st);
        if (e != cudaSuccess) return e;
        p.cols = (int)d.inner;
        p.rows = (int)d.hidden;
        p.xs = d.inner;
        p.ys = d.ys;
        p.x = h;
        p.w = wd;
        p.res = residual ? static_cast<const T*>(residual) + t * d.ys : nullptr;
        p.y = static_cast<T*>(y) + t * d.ys;
        e = few_tokens<T, false>(p, d.sms, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

// Few tokens, in groups that read the weights once each.  The products of gated_ffn.cu read 16-bit weights at one
// speed up to 128 tokens, but want fp32 ones split and odd rows copied first.  This file against that one, us:
//   bf16 2048 x 8192, in place      1 token 25 / 35, 2 30 / 35, 4 34 / 35, 8 (two groups) 65 / 35
//   fp16 4096 x 16384               1 token 70 / 86, 2 81 / 87, 4 (two groups) 160 / 87
//   bf16 2047 x 8191, copied        1 token 34 / 72, 4 49 / 72, 8 (two groups) 92 / 71
//   fp32 2048 x 8192                1 token 41 / 234, 8 (two groups) 88 / 216, 16 (four) 175 / 207
//   fp32 512 x 1408                 1 token 9 / 43, 8 19 / 43, 32 (four groups) 70 / 43
//   bf16, fp16 512 x 1408           1 token 9 / 14, 2 12 / 14, 4 12 / 14, 6 16 / 14, 8 18 / 14, 16 (two groups) 35 / 14
//   bf16 1024 x 4096                1 token 13 / 22, 2 15 / 23, 4 18 / 23, 6 24 / 23, 8 27 / 23
//   fp16 509 x 1371, copied         1 token 12 / 16, 2 15 / 17, 4 14 / 16, 6 18 / 17
bool gated_ffn_is_few(const gated_ffn_desc& d) {
    const bool f32 = d.dtype == CONV2D_F32;
    const int group = group_of(d);
    if (!group || d.tokens > (f32 ? 16 : 4)) return false;
    const bool copied = d.xs % 8 != 0 || d.hidden % 8 != 0 || d.inner % 8 != 0;
    return d.tokens <= (f32 || copied ? 2 : 1) * group;
}

int64_t gated_ffn_few_words(const gated_ffn_desc& d) { return group_of(d) * d.inner; }

cudaError_t launch_gated_ffn_few(const gated_ffn_desc& d, const void* x, const void* wg, const void* wu, const void* wd,
                                 const void* residual, void* y, float* saved, float* h, cudaStream_t st) {
    switch (d.dtype) {
        case CONV2D_F32: return run<float>(d, x, wg, wu, wd, residual, y, saved, h, st);
        case CONV2D_F16: return run<__half>(d, x, wg, wu, wd, residual, y, saved, h, st);
        default: return run<__nv_bfloat16>(d, x, wg, wu, wd, residual, y, saved, h, st);
    }
}

}  // namespace conv2d_gb300
