// Linear cross entropy of few tokens (serving, or the tail of a batch) on the
// CUDA cores: the pass over w is all there is, so w is read in
// place, whatever its type, row stride or alignment, and nothing is rounded
// below fp32 on the way (dz of a single token would be rounded as a whole).
//
// A warp takes four rows of w at a time, a vector slot a lane; h lies in shared
// memory, one column block per element of a vector, so that the lanes of a warp
// read consecutive words whatever the rows' offset from the 16-byte boundary
// (the four rows are a vector length apart and therefore offset alike; sixteen
// tokens take two rows, a single one two or four, see one_token_rows).  The 4 x
// tokens dot products are added over the warp together.
//   forward    each lane keeps the running (max, sum) of the products it ends
//              up with; blocks write one pair per token
//   backward   dz = g (exp(z - lse) - [v = y]) goes back to all lanes, which
//              write the four rows of dw = dz^T h and dz itself; a second
//              kernel reads w again, by columns, for dh = dz w
//
// Reading w bounds it up to four tokens: bf16 1 x 4096 x 65536 forward 85 us
// (6.3 TB/s), z and dw 170 us (6.3 TB/s), dh 100 us.  From eight tokens on it is
// h's way out of shared memory, four bytes a lane for four products: bf16 8 x 4096
// x 65536 forward 144 us, fp32 16 x 2048 x 50000 131 us (3.1 TB/s).
#include <type_traits>

#include "head_device.cuh"
#include "head_few.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512;
constexpr int kSmemMost = 200 * 1024;

struct FewParams {
    int tokens, hidden, vocab, reduction;
    int pitch;               // tokens between the blocks' parts
    int blocks;
    int64_t hs, ws, ignore;
    const void *h, *w;
    const int64_t* target;
    // forward
    float2* part;            // [blocks][pitch]
    float* z_target;
    // backward
    const float *lse, *dloss;
    void* dw;                // or null
    float* dz;               // [vocab][NT], or null
};

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T, int NT, int kRows, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 1) ce_few_kernel(const FewParams p) {
    constexpr int V = kVec<T>;
    constexpr int N = kRows * NT, kSpan = 32 / N, kOver = kSpan * NT;   // lanes per product and per row
    constexpr int P = kPair<NT>, NP = NT / P;
    using W = typename Word<P>::T;
    extern __shared__ __align__(16) float hs[];            // [NP][V][pitch][P]
    const W* words = reinterpret_cast<const W*>(hs);
    __shared__ float2 red[kThreads / 32][NT];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pitch = few_pitch<T>(p.hidden);
    for (int i = threadIdx.x; i < NT * V * pitch; i += kThreads) hs[i] = 0.f;
    __syncthreads();
    // This lane's token (k = r NT + t in lanes k kSpan on), its target and weight.
    const int mine_r = lane / kSpan / NT, mine_t = lane / kSpan % NT;
    int ty = -1;
    float g = 0.f, lse = 0.f;
    if (mine_t < p.tokens) {
        const int64_t t = p.target[mine_t];
        if (t != p.ignore && t >= 0 && t < p.vocab) ty = (int)t;
        if constexpr (BACKWARD) {
            lse = p.lse[mine_t];
            if (ty >= 0) {
                if (p.reduction == HEAD_REDUCE_NONE) {
                    g = p.dloss[mine_t];
                } else {
                    int count = 0;
                    for (int j = 0; j < p.tokens; ++j) {
                        const int64_t u = p.target[j];
                        count += u != p.ignore && u >= 0 && u < p.vocab;
                    }
                    g = p.reduction == HEAD_REDUCE_MEAN ? *p.dloss / (float)count : *p.dloss;
                }
            }
        }
    }
    for (int t = 0; t < p.tokens; ++t) {
        if constexpr (BACKWARD) {                          // rows without a target: zero, whatever they hold
            const int64_t y = p.target[t];
            if (y == p.ignore || y < 0 || y >= p.vocab) continue;
        }
        const T* h = static_cast<const T*>(p.h) + t * p.hs;
        for (int e = threadIdx.x; e < p.hidden; e += kThreads)
            hs[((t / P * V + (e & (V - 1))) * pitch + (e >> shift_bits<T>()) + 1) * P + t % P] = to_f32(h[e]);
    }
    __syncthreads();

    float m_run = -INFINITY, s_run = 0.f;
    // Four rows: a block of 4 V rows and an offset in it below V.
    const int quads = (int)(((int64_t)p.vocab + kRows * V - 1) / (kRows * V)) * V;
    for (int q = blockIdx.x * (kThreads / 32) + warp; q < quads; q += gridDim.x * (kThreads / 32)) {
        const int v0 = q / V * (kRows * V) + q % V;
        if (v0 >= p.vocab) continue;
        const T* w = static_cast<const T*>(p.w) + (int64_t)v0 * p.ws;
        const int shift = phase_of(w), slots = (p.hidden + shift + V - 1) >> shift_bits<T>();
        int off[V];
        word_offsets<T>(shift, pitch, off);
        W acc[kRows][NP];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int t = 0; t < NP; ++t) acc[r][t] = spread<P>(0.f);
        // Whole vectors of four whole rows first, so that nothing stands between
        // their loads; then the rows' ends (or all, at the end of the vocabulary).
        const bool four = v0 + (kRows - 1) * V < p.vocab;
        const int lo = shift != 0, hi = four ? max(lo, (p.hidden + shift) >> shift_bits<T>()) : lo;
        const auto add = [&](const Vec<T, V>(&raw)[kRows], int s) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                W f[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) f[r] = spread<P>(to_f32(raw[r].v[i]));
#pragma unroll
                for (int t = 0; t < NP; ++t) {
                    const W x = words[t * V * pitch + off[i] + s];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) acc[r][t] = fma_words(f[r], x, acc[r][t]);
                }
            }
        };
#pragma unroll(NT >= 8 ? 2 : 4)
        for (int s = lo + lane; s < hi; s += 32) {
            Vec<T, V> raw[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                raw[r] = *reinterpret_cast<const Vec<T, V>*>(w + (int64_t)r * V * p.ws + (s * V - shift));
            add(raw, s);
        }
        for (int j = lane; j < lo + slots - hi; j += 32) {
            const int s = j < lo ? j : hi + j - lo, e0 = s * V - shift;
            Vec<T, V> raw[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const bool in = v0 + r * V < p.vocab;
                raw[r] = load_part<T, V>(w + (in ? (int64_t)r * V * p.ws + e0 : 0), in ? max(0, -e0) : V,
                                         in ? min(V, p.hidden - e0) : 0);
            }
            add(raw, s);
        }
        float sums[N];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int t = 0; t < NP; ++t) {
                if constexpr (P == 2) unpack2f(acc[r][t], sums[r * NT + 2 * t], sums[r * NT + 2 * t + 1]);
                else sums[r] = acc[r][t];
            }
        const float z = warp_sums<N>(sums);
        const int v = v0 + mine_r * V;
        if constexpr (!BACKWARD) {
            if (v < p.vocab) {
                const float top = fmaxf(m_run, z), base = isinf(top) ? 0.f : top;
                s_run = s_run * exp2_of((m_run - base) * kLog2e) + exp2_of((z - base) * kLog2e);
                m_run = top;
                if (v == ty && lane % kSpan == 0) p.z_target[mine_t] = z;
            }
        } else {
            float d = 0.f;
            if (v < p.vocab && g != 0.f) d = (exp2_of((z - lse) * kLog2e) - (v == ty ? 1.f : 0.f)) * g;
            if (p.dz && v < p.vocab && lane % kSpan == 0) p.dz[(int64_t)v * NT + mine_t] = d;
            if (p.dw) {
                W dz[kRows][NP];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int t = 0; t < NP; ++t) {
                        const int k = r * NT + t * P;
                        const float a = __shfl_sync(0xffffffffu, d, k * kSpan);
                        if constexpr (P == 2) dz[r][t] = pack2f(a, __shfl_sync(0xffffffffu, d, (k + 1) * kSpan));
                        else dz[r][t] = a;
                    }
                // The rows of dw are contiguous; they may be offset unlike w's.
                T* out = static_cast<T*>(p.dw) + (int64_t)v0 * p.hidden;
                const int oshift = phase_of(out), oslots = (p.hidden + oshift + V - 1) >> shift_bits<T>();
                int ooff[V];
                word_offsets<T>(oshift, pitch, ooff);
                for (int s = lane; s < oslots; s += 32) {
                    const int e0 = s * V - oshift;
                    float o[kRows][V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        W sum[kRows];
#pragma unroll
                        for (int r = 0; r < kRows; ++r) sum[r] = spread<P>(0.f);
#pragma unroll
                        for (int t = 0; t < NP; ++t) {
                            const W x = words[t * V * pitch + ooff[i] + s];
#pragma unroll
                            for (int r = 0; r < kRows; ++r) sum[r] = fma_words(dz[r][t], x, sum[r]);
                        }
#pragma unroll
                        for (int r = 0; r < kRows; ++r) {
                            if constexpr (P == 2) o[r][i] = sum_halves(sum[r]);
                            else o[r][i] = sum[r];
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (v0 + r * V < p.vocab)
                            store_part<T, V>(out + (int64_t)r * V * p.hidden + e0, narrow<T, V>(o[r]), max(0, -e0),
                                             min(V, p.hidden - e0));
                }
            }
        }
    }
    if constexpr (!BACKWARD) {
        // Over the warp's rows, then over the warps.
#pragma unroll
        for (int o = kOver; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m_run, o), s2 = __shfl_xor_sync(0xffffffffu, s_run, o);
            const float top = fmaxf(m_run, m2), base = isinf(top) ? 0.f : top;
            s_run = s_run * exp2_of((m_run - base) * kLog2e) + s2 * exp2_of((m2 - base) * kLog2e);
            m_run = top;
        }
        if (lane < kOver && lane % kSpan == 0) red[warp][mine_t] = make_float2(m_run, s_run);
        __syncthreads();
        if (threadIdx.x < p.tokens) {
            float m = -INFINITY, s = 0.f;
            for (int k = 0; k < kThreads / 32; ++k) {
                const float2 o = red[k][threadIdx.x];
                const float top = fmaxf(m, o.x), base = isinf(top) ? 0.f : top;
                s = s * exp2_of((m - base) * kLog2e) + o.y * exp2_of((o.x - base) * kLog2e);
                m = top;
            }
            p.part[(int64_t)blockIdx.x * p.pitch + threadIdx.x] = make_float2(m, s);
        }
    }
}

// Elements lo .. hi-1 of a 16-byte vector, zero in the others' places.
__device__ __forceinline__ uint4 part_bits(const float* p, int lo, int hi) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = i >= lo && i < hi ? __float_as_uint(p[i]) : 0u;
    return make_uint4(b[0], b[1], b[2], b[3]);
}
template <typename T> __device__ __forceinline__ uint4 part_bits(const T* p, int lo, int hi) {
    uint32_t b[4] = {0u, 0u, 0u, 0u};
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= lo && i < hi) b[i / 2] |= (uint32_t)u[i] << (i % 2 * 16);
    return make_uint4(b[0], b[1], b[2], b[3]);
}

// Partial dh: a lane owns one vector of columns for all tokens, the warps of a
// block run down a share of w's rows (blockIdx.y), every `step`-th of them so
// that they are offset alike.  The share's dz lies in shared memory; the next
// four rows of w are on their way while four are added.  part [share][NT][lds].
constexpr int kDhThreads = 256, kDhWarps = kDhThreads / 32, kDhWords = 8192;
template <typename T, int NT>
__global__ void __launch_bounds__(kDhThreads, NT * kVec<T> <= 8 ? 4 : NT * kVec<T> <= 32 ? 3 : 2)
ce_few_dh_kernel(const T* w, int64_t ws, const float* dz, int hidden, int vocab, int step, int per, float* part,
                 int64_t lds) {
    constexpr int V = kVec<T>, kDeep = 4, P = kPair<NT>, NP = NT / P;
    using W = typename Word<P>::T;
    __shared__ __align__(16) float dzs[kDhWords];          // [rows of the share][NT]
    __shared__ float red[kDhWarps][32 * V];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.y / step * per + blockIdx.y % step, last = min(vocab, (int)(blockIdx.y / step + 1) * per);
    const int rows = last > first ? (last - first + step - 1) / step : 0;
    const int64_t row = (int64_t)step * ws;
    const int shift = phase_of(w + (int64_t)first * ws);
    const int64_t e0 = ((int64_t)blockIdx.x * 32 + lane) * V - shift;
    const int lo = e0 < 0 ? (int)-e0 : 0, hi = (int)max((int64_t)0, min((int64_t)V, hidden - e0));
    const T* base = w + (int64_t)first * ws + e0;
    for (int i = threadIdx.x; i < rows * NT; i += kDhThreads) dzs[i] = dz[((int64_t)first + i / NT * step) * NT + i % NT];
    W acc[NP][V];
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[t][i] = spread<P>(0.f);
    const auto add = [&](const uint4& bits, int j) {
        f32x2 two[V / 2];
        Pairs<T>::widen(bits, two);
        float x[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack2f(two[i], x[2 * i], x[2 * i + 1]);
        W d[NP];
#pragma unroll
        for (int t = 0; t < NP; ++t) d[t] = reinterpret_cast<const W*>(dzs)[j * NP + t];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const W f = spread<P>(x[i]);
#pragma unroll
            for (int t = 0; t < NP; ++t) acc[t][i] = fma_words(d[t], f, acc[t][i]);
        }
    };
    const int mine = rows > warp ? (rows - warp + kDhWarps - 1) / kDhWarps : 0, groups = mine / kDeep;
    __syncthreads();
    const auto run = [&](auto ends) {                      // ends: some lane's vector reaches past its row
        const auto fetch = [&](int j) {
            const T* at = base + (int64_t)j * row;
            if constexpr (decltype(ends)::value) {
                return part_bits(at, lo, hi);
            } else {
                return *reinterpret_cast<const uint4*>(at);
            }
        };
        uint4 now[kDeep], next[kDeep];
        if (groups) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) now[k] = fetch(warp + k * kDhWarps);
        }
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            const int j = warp + g * kDeep * kDhWarps;
            if (g + 1 < groups) {
#pragma unroll
                for (int k = 0; k < kDeep; ++k) next[k] = fetch(j + (kDeep + k) * kDhWarps);
            }
#pragma unroll
            for (int k = 0; k < kDeep; ++k) add(now[k], j + k * kDhWarps);
#pragma unroll
            for (int k = 0; k < kDeep; ++k) now[k] = next[k];
        }
        for (int j = warp + groups * kDeep * kDhWarps; j < rows; j += kDhWarps) add(fetch(j), j);
    };
    if (__all_sync(0xffffffffu, lo == 0 && hi == V)) run(std::false_type{});
    else run(std::true_type{});
    // Over the warps, a token at a time.
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t) __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (P == 2) {
                float a, b;
                unpack2f(acc[t / 2][i], a, b);
                red[warp][i * 32 + lane] = t % 2 ? b : a;
            } else {
                red[warp][i * 32 + lane] = acc[t][i];
            }
        }
        __syncthreads();
        if (threadIdx.x < 32 * V) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kDhWarps; ++k) sum += red[k][(threadIdx.x % V) * 32 + threadIdx.x / V];
            const int64_t e = (int64_t)blockIdx.x * 32 * V + threadIdx.x - shift;
            if (e >= 0 && e < hidden) part[((int64_t)blockIdx.y * NT + t) * lds + e] = sum;
        }
    }
}

// dh from the partial sums: 32 columns a block, eight threads a column.
template <typename T>
__global__ void __launch_bounds__(256) ce_few_join_kernel(const float* part, int shares, int nt, int hidden, int64_t lds,
                                                          T* dh) {
    __shared__ float red[8][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, k0 = threadIdx.x >> 5, t = blockIdx.y;
    const int c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < hidden) {
#pragma unroll 8
        for (int k = k0; k < shares; k += 8) sum += part[((int64_t)k * nt + t) * lds + c];
    }
    red[k0][lane] = sum;
    __syncthreads();
    if (k0 == 0 && c < hidden) {
#pragma unroll
        for (int k = 1; k < 8; ++k) sum += red[k][lane];
        dh[(int64_t)t * hidden + c] = from_f32<T>(sum);
    }
}

int nt_of(int64_t tokens) { return tokens <= 1 ? 1 : tokens <= 2 ? 2 : tokens <= 4 ? 4 : tokens <= 8 ? 8 : 16; }

template <typename T> size_t few_smem(int64_t tokens, int64_t hidden) {
    return (size_t)nt_of(tokens) * kVec<T> * few_pitch<T>((int)hidden) * sizeof(float);
}
bool few_fits(const linear_ce_desc& d, int64_t tokens) {
    return (d.dtype == CONV2D_F32 ? few_smem<float>(tokens, d.hidden) : few_smem<__half>(tokens, d.hidden)) <=
           (size_t)kSmemMost;
}

template <typename T, int NT, int ROWS, bool BACKWARD> cudaError_t few_launch(const FewParams& p, cudaStream_t st) {
    const size_t smem = few_smem<T>(NT, p.hidden);
    const cudaError_t e = allow_smem(ce_few_kernel<T, NT, ROWS, BACKWARD>, kSmemMost);
    if (e != cudaSuccess) return e;
    return launch_after(ce_few_kernel<T, NT, ROWS, BACKWARD>, dim3((unsigned)p.blocks), dim3(kThreads), smem,
                        st, p);
}

// Rows of w that a warp takes at a time for a single token: two or four, by the
// turns of the warp that has most of them.  A turn costs its rows' bytes and, for the
// trip to memory and the sum over the warp, as much as another 768.  Two rows / four,
// bf16, forward (dw goes the same way):
//   256 features    32000 rows 12.4 / 10.4 us, 131072 rows 30.9 / 21.8, 2000 rows 4.7 / 5.0
//   1024 features   5000 rows 10.4 / 9.7, 10007 rows 12.4 / 16.0, 50257 rows 24.0 / 27.9
//   2487 features   64640 rows 63.7 / 58.7;   4096   10007 rows 27.3 / 42.5
// The rule is at most 2.5 % behind the better one at the 36 shapes measured.
int one_token_rows(int64_t vocab, int64_t row_bytes, int vec, int blocks) {
    const int64_t warps = (int64_t)blocks * (kThreads / 32);
    const auto cost = [&](int64_t rows) {
        const int64_t groups = (vocab + rows * vec - 1) / (rows * vec) * vec;
        return (groups + warps - 1) / warps * (rows * row_bytes + 768);
    };
    return cost(2) <= cost(4) ? 2 : 4;
}
template <typename T, bool BACKWARD> cudaError_t few_tokens(const FewParams& p, cudaStream_t st) {
    switch (nt_of(p.tokens)) {
        case 1:
            return one_token_rows(p.vocab, p.hidden * (int64_t)sizeof(T), kVec<T>, p.blocks) == 2
                       ? few_launch<T, 1, 2, BACKWARD>(p, st)
                       : few_launch<T, 1, 4, BACKWARD>(p, st);
        case 2: return few_launch<T, 2, 4, BACKWARD>(p, st);
        case 4: return few_launch<T, 4, 4, BACKWARD>(p, st);
        case 8: return few_launch<T, 8, 4, BACKWARD>(p, st);
    }
    if constexpr (sizeof(T) == 4) {
        return few_launch<T, 16, 2, BACKWARD>(p, st);
    } else {
        return cudaErrorInvalidValue;
    }
}
template <bool BACKWARD> cudaError_t few(const linear_ce_desc& d, const FewParams& p, cudaStream_t st) {
    switch (d.dtype) {
        case CONV2D_F32: return few_tokens<float, BACKWARD>(p, st);
        case CONV2D_F16: return few_tokens<__half, BACKWARD>(p, st);
        default: return few_tokens<__nv_bfloat16, BACKWARD>(p, st);
    }
}

// Rows a warp of the dh kernel steps over, and the shares: four blocks an SM, at
// least 32 rows each and no more than its shared memory takes.
struct DhPlan { int step, per, shares, columns; };
DhPlan dh_plan(const linear_ce_desc& d) {
    DhPlan p;
    const int64_t V = 16 / (int64_t)elem_bytes(d.dtype);
    p.step = d.ws % V == 0 ? 1 : (int)V;
    p.columns = (int)((d.hidden + (V - 1) + 32 * V - 1) / (32 * V));    // rows may begin V - 1 elements into a vector
    int64_t ranges = (4 * d.sms + p.columns * p.step - 1) / (p.columns * p.step);
    const int64_t most = (d.vocab + 32 * p.step - 1) / (32 * p.step);
    if (ranges > most) ranges = most;
    const int64_t room = kDhWords / nt_of(d.tokens) * p.step, least = (d.vocab + room - 1) / room;
    if (ranges < least) ranges = least;
    p.per = (int)((d.vocab + ranges - 1) / ranges);
    p.shares = (int)((d.vocab + p.per - 1) / p.per) * p.step;
    return p;
}

template <typename T> cudaError_t dh_typed(const linear_ce_desc& d, const void* w, const float* dz, float* sums, void* dh, cudaStream_t st) {
    const DhPlan pl = dh_plan(d);
    const int nt = nt_of(d.tokens);
    auto kern = nt == 1   ? ce_few_dh_kernel<T, 1>
                : nt == 2 ? ce_few_dh_kernel<T, 2>
                : nt == 4 ? ce_few_dh_kernel<T, 4>
                          : ce_few_dh_kernel<T, 8>;
    if constexpr (sizeof(T) == 4) {
        if (nt == 16) kern = ce_few_dh_kernel<T, 16>;
    }
    // As many whole ranges of rows a launch as the grid's y numbers shares of (one
    // launch up to 33 million rows; share numbers past it would cost the kernel
    // registers, 1 to 4 %).
    const int most = 65535 / pl.step * pl.step;
    for (int s = 0; s < pl.shares; s += most) {
        const int64_t row = (int64_t)(s / pl.step) * pl.per;
        const int n = pl.shares - s < most ? pl.shares - s : most;
        const cudaError_t e = launch_after(kern, dim3((unsigned)pl.columns, (unsigned)n), dim3(kDhThreads), 0, st,
                                           static_cast<const T*>(w) + row * d.ws, d.ws, dz + row * nt, (int)d.hidden,
                                           (int)(d.vocab - row), pl.step, pl.per, sums + (int64_t)s * nt * d.hidden,
                                           d.hidden);
        if (e != cudaSuccess) return e;
    }
    return launch_after(ce_few_join_kernel<T>, dim3((unsigned)((d.hidden + 31) / 32), (unsigned)d.tokens), dim3(256), 0, st,
                        sums, pl.shares, nt, (int)d.hidden, d.hidden, static_cast<T*>(dh));
}

}  // namespace

// Few tokens, whose h fits a block's shared memory.  The products of
// linear_ce.cu read w at one speed whatever the tokens, but want fp32 split and
// odd rows copied first.  Forward / backward, this file against that one:
//   bf16 4096 x 65536, in place   4 tokens  94 / 321 us, 132 / 338;   8 tokens 144 / 447, 109 / 406
//   bf16 2487 x 64640, copied     8 tokens 114 / 327 us, 211 / 465
//   fp32 2048 x 50000             8 tokens  81 / 249 us, 516 / 825;  16 tokens 131 / 394, 411 / 769
//   fp32 1024 x 50000            32 tokens 218 / 604 us (a form for 32 at once), 203 / 414
// Forward of fp32 takes up to 32 tokens in groups, each of which reads w again:
// 32 x 2048 x 50000 257 us, 415 on the tensor cores; 20 x 3900 x 9472 116, 195; 32 x
// 256 x 9472 25, 27; behind only where rows are a tile wide: 32 x 100 x 50000 44, 38.
bool linear_ce_is_few(const linear_ce_desc& d, bool backward) {
    if (d.dtype == CONV2D_F32 && !backward) return d.tokens <= 32 && few_fits(d, d.tokens < 8 ? d.tokens : 8);
    const bool copied = d.hs % 8 != 0 || d.ws % 8 != 0;
    return d.tokens <= (d.dtype == CONV2D_F32 ? 16 : copied ? 8 : 4) && few_fits(d, d.tokens);
}

// fp32 words of dz and of the partial sums of dh.
int64_t linear_ce_few_dz(const linear_ce_desc& d) { return d.vocab * nt_of(d.tokens); }
int64_t linear_ce_few_sums(const linear_ce_desc& d) { return (int64_t)dh_plan(d).shares * nt_of(d.tokens) * d.hidden; }

cudaError_t launch_ce_few_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target, void* part,
                              float* z_target, cudaStream_t st) {
    const int64_t most = d.tokens <= 8 || !few_fits(d, 16) ? 8 : 16;
    for (int64_t t = 0; t < d.tokens; t += most) {
        FewParams p{};
        p.tokens = (int)(d.tokens - t < most ? d.tokens - t : most);
        p.pitch = (int)d.tokens;
        p.blocks = linear_ce_few_blocks(d);
        p.hidden = (int)d.hidden; p.vocab = (int)d.vocab; p.reduction = d.reduction;
        p.hs = d.hs; p.ws = d.ws; p.ignore = d.ignore_index;
        p.h = static_cast<const uint8_t*>(h) + (size_t)(t * d.hs) * elem_bytes(d.dtype);
        p.w = w;
        p.target = target + t;
        p.part = static_cast<float2*>(part) + t;
        p.z_target = z_target + t;
        const cudaError_t e = few<false>(d, p, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_ce_few_bwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                              const float* lse, const float* dloss, void* dh, void* dw, float* dz, float* sums,
                              cudaStream_t st) {
    FewParams p{};
    p.tokens = (int)d.tokens; p.hidden = (int)d.hidden; p.vocab = (int)d.vocab; p.reduction = d.reduction;
    p.blocks = linear_ce_few_blocks(d);
    p.hs = d.hs; p.ws = d.ws; p.ignore = d.ignore_index;
    p.h = h; p.w = w; p.target = target;
    p.lse = lse; p.dloss = dloss; p.dw = dw;
    p.dz = dh ? dz : nullptr;
    const cudaError_t e = few<true>(d, p, st);
    if (e != cudaSuccess || !dh) return e;
    switch (d.dtype) {
        case CONV2D_F32: return dh_typed<float>(d, w, dz, sums, dh, st);
        case CONV2D_F16: return dh_typed<__half>(d, w, dz, sums, dh, st);
        default: return dh_typed<__nv_bfloat16>(d, w, dz, sums, dh, st);
    }
}

}  // namespace conv2d_gb300
