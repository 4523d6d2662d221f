// Linear cross entropy of at most eight tokens (serving, or the tail of a
// batch) on the CUDA cores: the pass over w is all there is, so w is read in
// place, whatever its type, row stride or alignment, and nothing is rounded
// below fp32 on the way (dz of a single token would be rounded as a whole).
//
// A warp takes four rows of w at a time, a vector slot a lane; h lies in shared
// memory, one column block per element of a vector, so that the lanes of a warp
// read consecutive words whatever the rows' offset from the 16-byte boundary
// (the four rows are a vector length apart and therefore offset alike).  The
// 4 x tokens dot products are added over the warp together.
//   forward    each lane keeps the running (max, sum) of the products it ends
//              up with; blocks write one pair per token
//   backward   dz = g (exp(z - lse) - [v = y]) goes back to all lanes, which
//              write the four rows of dw = dz^T h and dz itself; a second
//              kernel reads w again, by columns, for dh = dz w
#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512, kRows = 4;
constexpr int kSmemMost = 200 * 1024;

struct FewParams {
    int tokens, hidden, vocab, reduction;
    int64_t hs, ws, ignore;
    const void *h, *w;
    const int64_t* target;
    // forward
    float2* part;            // [blocks][tokens]
    float* z_target;
    // backward
    const float *lse, *dloss;
    void* dw;                // or null
    float* dz;               // [tokens][vocab]
    float* one;              // set to 1 (the scale of the joined sums of dh)
};

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T> __host__ __device__ constexpr int shift_bits() { return sizeof(T) == 4 ? 2 : 3; }

// Words of h per token in shared memory: for each element of a vector, one
// column block of slots with a zero slot on both sides.
template <typename T> __host__ __device__ int few_pitch(int hidden) {
    return ((hidden + 16 / (int)sizeof(T) - 1) >> shift_bits<T>()) + 3;
}

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __device__ __forceinline__ int phase_of(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// Offsets of the V elements of slot 0 in a token's words, for rows that start
// `shift` elements after a boundary: element i of slot s is h's element
// s V + i - shift.
template <typename T> __device__ __forceinline__ void word_offsets(int shift, int pitch, int (&off)[kVec<T>]) {
    constexpr int V = kVec<T>;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i - shift;                           // -(V-1) .. V-1
        off[i] = (e & (V - 1)) * pitch + (e >> shift_bits<T>()) + 1;
    }
}

template <typename T, int NT, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 1) ce_few_kernel(const FewParams p) {
    constexpr int V = kVec<T>, N = kRows * NT, kSpan = 32 / N;     // lanes per product
    extern __shared__ float hs[];                          // [NT][V][pitch]
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
            hs[(t * V + (e & (V - 1))) * pitch + (e >> shift_bits<T>()) + 1] = to_f32(h[e]);
    }
    if (BACKWARD && blockIdx.x == 0 && threadIdx.x == 0) *p.one = 1.f;
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
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.f;
#pragma unroll 2
        for (int s = lane; s < slots; s += 32) {
            const int e0 = s * V - shift;
            Vec<T, V> raw[kRows];
            const bool whole = e0 >= 0 && e0 + V <= p.hidden;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (whole && v0 + r * V < p.vocab)
                    raw[r] = *reinterpret_cast<const Vec<T, V>*>(w + (int64_t)r * V * p.ws + e0);
            if (!whole || v0 + (kRows - 1) * V >= p.vocab) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const bool in = v0 + r * V < p.vocab;
                    if (!whole || !in)
                        raw[r] = load_part<T, V>(w + (in ? (int64_t)r * V * p.ws + e0 : 0), in ? max(0, -e0) : V,
                                                 in ? min(V, p.hidden - e0) : 0);
                }
            }
            float f[kRows][V];
#pragma unroll
            for (int r = 0; r < kRows; ++r) widen(raw[r], f[r]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = hs[t * V * pitch + off[i] + s];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) acc[r * NT + t] = fmaf(f[r][i], x, acc[r * NT + t]);
                }
            }
        }
        const float z = warp_sums<N>(acc);
        const int v = v0 + mine_r * V;
        if constexpr (!BACKWARD) {
            if (v < p.vocab) {
                const float top = fmaxf(m_run, z), base = top == -INFINITY ? 0.f : top;
                s_run = s_run * exp2_of((m_run - base) * kLog2e) + exp2_of((z - base) * kLog2e);
                m_run = top;
                if (v == ty && lane % kSpan == 0) p.z_target[mine_t] = z;
            }
        } else {
            float d = 0.f;
            if (v < p.vocab && g != 0.f) d = (exp2_of((z - lse) * kLog2e) - (v == ty ? 1.f : 0.f)) * g;
            if (v < p.vocab && mine_t < p.tokens && lane % kSpan == 0) p.dz[(int64_t)mine_t * p.vocab + v] = d;
            if (p.dw) {
                float dz[N];
#pragma unroll
                for (int k = 0; k < N; ++k) dz[k] = __shfl_sync(0xffffffffu, d, k * kSpan);
                // The rows of dw are contiguous; they may be offset unlike w's.
                T* out = static_cast<T*>(p.dw) + (int64_t)v0 * p.hidden;
                const int oshift = phase_of(out), oslots = (p.hidden + oshift + V - 1) >> shift_bits<T>();
                int ooff[V];
                word_offsets<T>(oshift, pitch, ooff);
                for (int s = lane; s < oslots; s += 32) {
                    const int e0 = s * V - oshift;
                    float o[kRows][V];
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
#pragma unroll
                        for (int i = 0; i < V; ++i) o[r][i] = 0.f;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float x = hs[t * V * pitch + ooff[i] + s];
#pragma unroll
                            for (int r = 0; r < kRows; ++r) o[r][i] = fmaf(dz[r * NT + t], x, o[r][i]);
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
        // Over the warp's four rows (8 and 16 lanes apart), then over the warps.
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m_run, o), s2 = __shfl_xor_sync(0xffffffffu, s_run, o);
            const float top = fmaxf(m_run, m2), base = top == -INFINITY ? 0.f : top;
            s_run = s_run * exp2_of((m_run - base) * kLog2e) + s2 * exp2_of((m2 - base) * kLog2e);
            m_run = top;
        }
        if (lane < 8 && lane % kSpan == 0) red[warp][mine_t] = make_float2(m_run, s_run);
        __syncthreads();
        if (threadIdx.x < p.tokens) {
            float m = -INFINITY, s = 0.f;
            for (int k = 0; k < kThreads / 32; ++k) {
                const float2 o = red[k][threadIdx.x];
                const float top = fmaxf(m, o.x), base = top == -INFINITY ? 0.f : top;
                s = s * exp2_of((m - base) * kLog2e) + o.y * exp2_of((o.x - base) * kLog2e);
                m = top;
            }
            p.part[(int64_t)blockIdx.x * p.tokens + threadIdx.x] = make_float2(m, s);
        }
    }
}

// Partial dh: a thread owns one vector of columns for all tokens and runs down
// a share of w's rows (blockIdx.y), every `step`-th of them so that they are
// offset alike.  part [share][tokens][lds].
template <typename T, int NT>
__global__ void __launch_bounds__(128) ce_few_dh_kernel(const T* w, int64_t ws, const float* dz, int tokens, int hidden,
                                                        int vocab, int step, int per, float* part, int64_t lds) {
    constexpr int V = kVec<T>;
    pdl_wait();
    const int first = blockIdx.y / step * per + blockIdx.y % step;
    const int last = min(vocab, (int)(blockIdx.y / step + 1) * per);
    const int shift = phase_of(w + (int64_t)first * ws);
    const int64_t e0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V - shift;
    if (e0 >= hidden) return;
    const int lo = e0 < 0 ? (int)-e0 : 0, hi = (int)min((int64_t)V, hidden - e0);
    float acc[NT][V];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[t][i] = 0.f;
#pragma unroll 4
    for (int v = first; v < last; v += step) {
        float f[V];
        widen(load_part<T, V>(w + (int64_t)v * ws + e0, lo, hi), f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t < tokens) {
                const float d = __ldg(dz + (int64_t)t * vocab + v);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[t][i] = fmaf(d, f[i], acc[t][i]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t < tokens) {
            float* out = part + ((int64_t)blockIdx.y * tokens + t) * lds + e0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= lo && i < hi) out[i] = acc[t][i];
        }
    }
}

int nt_of(int64_t tokens) { return tokens <= 1 ? 1 : tokens <= 2 ? 2 : tokens <= 4 ? 4 : 8; }

template <typename T> size_t few_smem(const linear_ce_desc& d) {
    return (size_t)nt_of(d.tokens) * kVec<T> * few_pitch<T>((int)d.hidden) * sizeof(float);
}

template <typename T, int NT, bool BACKWARD> cudaError_t few_launch(const linear_ce_desc& d, const FewParams& p, cudaStream_t st) {
    const size_t smem = few_smem<T>(d);
    const cudaError_t e = cudaFuncSetAttribute(ce_few_kernel<T, NT, BACKWARD>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(ce_few_kernel<T, NT, BACKWARD>, dim3((unsigned)linear_ce_few_blocks()), dim3(kThreads), smem, st,
                        p);
}
template <typename T, bool BACKWARD> cudaError_t few_tokens(const linear_ce_desc& d, const FewParams& p, cudaStream_t st) {
    switch (nt_of(d.tokens)) {
        case 1: return few_launch<T, 1, BACKWARD>(d, p, st);
        case 2: return few_launch<T, 2, BACKWARD>(d, p, st);
        case 4: return few_launch<T, 4, BACKWARD>(d, p, st);
        default: return few_launch<T, 8, BACKWARD>(d, p, st);
    }
}
template <bool BACKWARD> cudaError_t few(const linear_ce_desc& d, const FewParams& p, cudaStream_t st) {
    switch (d.dtype) {
        case CONV2D_F32: return few_tokens<float, BACKWARD>(d, p, st);
        case CONV2D_F16: return few_tokens<__half, BACKWARD>(d, p, st);
        default: return few_tokens<__nv_bfloat16, BACKWARD>(d, p, st);
    }
}

// Rows a thread of the dh kernel skips, and the shares: enough blocks for four
// an SM, at least 32 rows each.
struct DhPlan { int step, per, shares; };
DhPlan dh_plan(const linear_ce_desc& d) {
    DhPlan p;
    const int64_t V = 16 / (int64_t)elem_bytes(d.dtype);
    p.step = d.ws % V == 0 ? 1 : (int)V;
    const int64_t gx = ((d.hidden + V - 1 + V - 1) / V + 127) / 128;
    int64_t ranges = (4 * device_sm_count() + gx * p.step - 1) / (gx * p.step);
    const int64_t most = (d.vocab + 32 * p.step - 1) / (32 * p.step);
    if (ranges > most) ranges = most;
    if (ranges > 128) ranges = 128;
    if (ranges < 1) ranges = 1;
    p.per = (int)((d.vocab + ranges - 1) / ranges);
    p.shares = (int)((d.vocab + p.per - 1) / p.per) * p.step;
    return p;
}

template <typename T> cudaError_t dh_typed(const linear_ce_desc& d, const void* w, const float* dz, float* sums, int64_t lds,
                                           cudaStream_t st) {
    const DhPlan pl = dh_plan(d);
    constexpr int V = kVec<T>;
    const dim3 grid((unsigned)(((d.hidden + V - 1 + V - 1) / V + 127) / 128), (unsigned)pl.shares);
    auto kern = nt_of(d.tokens) == 1   ? ce_few_dh_kernel<T, 1>
                : nt_of(d.tokens) == 2 ? ce_few_dh_kernel<T, 2>
                : nt_of(d.tokens) == 4 ? ce_few_dh_kernel<T, 4>
                                       : ce_few_dh_kernel<T, 8>;
    return launch_after(kern, grid, dim3(128), 0, st, static_cast<const T*>(w), d.ws, dz, (int)d.tokens, (int)d.hidden,
                        (int)d.vocab, pl.step, pl.per, sums, lds);
}

}  // namespace

int linear_ce_few_blocks() { return device_sm_count(); }

// At most eight tokens whose h fits a block's shared memory.
bool linear_ce_is_few(const linear_ce_desc& d) {
    if (d.tokens > 8) return false;
    const size_t smem = d.dtype == CONV2D_F32 ? few_smem<float>(d) : few_smem<__half>(d);
    return smem <= (size_t)kSmemMost;
}

int linear_ce_few_shares(const linear_ce_desc& d) { return dh_plan(d).shares; }

cudaError_t launch_ce_few_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target, void* part,
                              float* z_target, cudaStream_t st) {
    FewParams p{};
    p.tokens = (int)d.tokens; p.hidden = (int)d.hidden; p.vocab = (int)d.vocab; p.reduction = d.reduction;
    p.hs = d.hs; p.ws = d.ws; p.ignore = d.ignore_index;
    p.h = h; p.w = w; p.target = target;
    p.part = static_cast<float2*>(part);
    p.z_target = z_target;
    return few<false>(d, p, st);
}

cudaError_t launch_ce_few_bwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                              const float* lse, const float* dloss, void* dw, float* dz, float* one, bool want_dh,
                              float* sums, int64_t lds, cudaStream_t st) {
    FewParams p{};
    p.tokens = (int)d.tokens; p.hidden = (int)d.hidden; p.vocab = (int)d.vocab; p.reduction = d.reduction;
    p.hs = d.hs; p.ws = d.ws; p.ignore = d.ignore_index;
    p.h = h; p.w = w; p.target = target;
    p.lse = lse; p.dloss = dloss; p.dw = dw; p.dz = dz; p.one = one;
    cudaError_t e = few<true>(d, p, st);
    if (e != cudaSuccess || !want_dh) return e;
    switch (d.dtype) {
        case CONV2D_F32: return dh_typed<float>(d, w, dz, sums, lds, st);
        case CONV2D_F16: return dh_typed<__half>(d, w, dz, sums, lds, st);
        default: return dh_typed<__nv_bfloat16>(d, w, dz, sums, lds, st);
    }
}

}  // namespace conv2d_gb300
