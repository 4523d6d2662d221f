// Layer norm over rows of adjacent elements, forward and backward.
//
// Forward: a row belongs to `tpr` threads of one block (a power of two up to a
// warp, or whole warps), or to a cluster of up to eight blocks.  Each thread
// keeps its part of the row in registers, so x is read once: the mean is
// summed first and the squares of x - mean second (no cancellation between
// large sums), then y is written.
//
// Backward: dx needs two sums over the row, sum a and sum a z (a = dy gamma,
// z = (x - mean) rstd); dgamma and dbeta are sums over rows.  Rows are dealt
// out to a fixed grid, every thread keeps the same columns for all of its
// rows and adds dy z and dy into registers; the blocks' sums go through the
// workspace to a second kernel that adds them in a fixed order.  Rows longer
// than a block's registers hold take two passes over x and dy instead.
//
// Rows are cut into 16-byte vectors at the memory's own 16-byte boundaries, so
// rows that start off a boundary (odd strides) still move in full vectors,
// with single elements only at the two ends.  That needs all tensors of a call
// to sit alike against the boundary; otherwise elements move one by one.
#include <cooperative_groups.h>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace cg = cooperative_groups;

namespace {

struct LnParams {
    int64_t rows, xs, ys;
    int cols;
    int tpr;             // threads per row: a power of two below 32, or a multiple of 32
    int cs;              // blocks (one cluster) per row; above 1: tpr = the block's threads
    int per_block;       // vector slots of a row per block of the cluster
    int groups;          // backward: row groups of the grid (rows in flight)
    int param_f32;
    int cut_alike;       // backward: every row starts at the same place after a 16-byte boundary
    int vec_params;      // gamma and beta rows are 16-byte aligned like the data's vectors
    float eps, inv_cols;
    const void *x, *dy, *gamma, *beta;
    void *y, *dx;        // y may be x: no __restrict__
    float *mean, *rstd;
    const float *mean_in, *rstd_in;
    float *part;         // backward: [parts][2][cols] sums of dy z and dy
    int want_params;
};

// How a call's rows are cut: whole 16-byte vectors only; vectors with single
// elements at a row's ends; single elements.  (Whole rows get kernels of their
// own: the code for the ends costs the backward kernel its registers.)
enum Cut { WHOLE = 0, ENDS = 1, SINGLE = 2 };
template <typename T, int CUT> __host__ __device__ constexpr int vec_of() { return CUT == SINGLE ? 1 : 16 / (int)sizeof(T); }

// Vector slot s of a row that starts `shift` elements after a 16-byte boundary
// covers elements [s V - shift, s V - shift + V); only the row's first and
// last slot can stick out of it.
template <int V> __device__ __forceinline__ bool slot_whole(int64_t e0, int cols) { return e0 >= 0 && e0 + V <= cols; }

// A slot's elements that lie in the row: [first, last).
template <int CUT> __device__ __forceinline__ int slot_first(int64_t e0) { return CUT == ENDS && e0 < 0 ? (int)-e0 : 0; }
template <int CUT, int V> __device__ __forceinline__ int slot_last(int64_t e0, int cols) {
    return CUT == ENDS && e0 + V > cols ? (int)(cols - e0) : V;
}

// NV slots s0 + j * step of a row, those below s1.  The whole ones first, so
// that all of their loads are issued before the rare partial ones branch.
template <typename T, int CUT, int V, int NV>
__device__ __forceinline__ void load_row(const T* x, int cols, int shift, int s0, int step, int s1, Vec<T, V> (&raw)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = s0 + j * step, e0 = s * V - shift;
        if (s < s1 && (CUT != ENDS || slot_whole<V>(e0, cols))) raw[j] = *reinterpret_cast<const Vec<T, V>*>(x + e0);
    }
    if (CUT == ENDS) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int s = s0 + j * step, e0 = s * V - shift;
            if (s < s1 && !slot_whole<V>(e0, cols)) raw[j] = load_part<T, V>(x + e0, slot_first<CUT>(e0), slot_last<CUT, V>(e0, cols));
        }
    }
}

// Sum over the tpr threads of each row group (red: 32 floats, one per warp).
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
    v = lane_sum(v, tpr < 32 ? tpr : 32);
    if (tpr <= 32) return v;
    const int wpr = tpr >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    const int first = warp / wpr * wpr;
    return lane_sum(lane < wpr ? red[first + lane] : 0.f, 32);
}

// H pairs or single values of a vector slot, as the arithmetic takes them.
template <typename T, int V> struct Values {
    static constexpr int H = V / 2;
    f32x2 v[H];
    __device__ __forceinline__ void widen(const Vec<T, V>& a) {
        Pairs<T>::widen(*reinterpret_cast<const uint4*>(&a), v);
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = pack2f(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void keep(int lo, int hi) {         // zero outside [lo, hi)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float a, b;
            unpack2f(v[i], a, b);
            v[i] = pack2f(2 * i >= lo && 2 * i < hi ? a : 0.f, 2 * i + 1 >= lo && 2 * i + 1 < hi ? b : 0.f);
        }
    }
    __device__ __forceinline__ void minus(float m) {
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = add2(v[i], both(-m));
    }
    __device__ __forceinline__ float sum() const {
        f32x2 s = v[0];
#pragma unroll
        for (int i = 1; i < H; ++i) s = add2(s, v[i]);
        return sum_halves(s);
    }
    __device__ __forceinline__ float squares() const {
        f32x2 s = mul2(v[0], v[0]);
#pragma unroll
        for (int i = 1; i < H; ++i) s = fma2(v[i], v[i], s);
        return sum_halves(s);
    }
    __device__ __forceinline__ Vec<T, V> affine(float r, const Values& g, const Values& b) const {
        f32x2 o[H];
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = fma2(mul2(v[i], both(r)), g.v[i], b.v[i]);
        const uint4 w = Pairs<T>::narrow(o);
        return *reinterpret_cast<const Vec<T, V>*>(&w);
    }
};
template <typename T> struct Values<T, 1> {
    float v;
    __device__ __forceinline__ void widen(const Vec<T, 1>& a) { v = to_f32(a.v[0]); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = f[0]; }
    __device__ __forceinline__ void keep(int, int) {}
    __device__ __forceinline__ void minus(float m) { v -= m; }
    __device__ __forceinline__ float sum() const { return v; }
    __device__ __forceinline__ float squares() const { return v * v; }
    __device__ __forceinline__ Vec<T, 1> affine(float r, const Values& g, const Values& b) const {
        Vec<T, 1> o;
        o.v[0] = from_f32<T>(fmaf(v * r, g.v, b.v));
        return o;
    }
};

// Forward in registers: one read of x, one write of y.  A row takes as few
// threads as keep every row's threads on the GPU at once, so small calls are
// bound by one trip to memory and two exchanges (one row of 4096 bf16 2.7 us,
// 2.0 of them launch), and 65536 x 64 bf16 takes 5.7 us.  A few very long rows
// go to clusters: 32 x 200704 fp16 12.8 us (2.0 TB/s), where 128 blocks are what
// 32 rows in clusters of four give.
template <typename T, int CUT, int NV>
__global__ void __launch_bounds__(1024) layernorm_fwd_kernel(const LnParams p) {
    constexpr int V = vec_of<T, CUT>();
    constexpr bool EARLY = NV == 1;                    // one vector a thread: gamma and beta ride with x's latency
    __shared__ float red[2][32];
    __shared__ float4 share;
    pdl_wait();
    const int rpb = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr, t = threadIdx.x - sub * p.tpr;
    const int rank = p.cs > 1 ? (int)(blockIdx.x % p.cs) : 0;
    const int64_t row = (int64_t)(blockIdx.x / p.cs) * rpb + sub;
    const bool live = row < p.rows;
    const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.xs;
    T* y = static_cast<T*>(p.y) + (live ? row : 0) * p.ys;
    const int shift = CUT != ENDS ? 0 : (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int slots = live ? (p.cols + shift + V - 1) / V : 0;
    const int s0 = rank * p.per_block + t, s1 = min(slots, rank * p.per_block + p.per_block);
    const bool vec = p.vec_params && shift == 0;

    Vec<T, V> raw[NV];
    load_row<T, CUT, V, NV>(x, p.cols, shift, s0, p.tpr, s1, raw);
    Values<T, V> g, b;
    auto params = [&](int e0) {
        const int lo = slot_first<CUT>(e0), hi = slot_last<CUT, V>(e0, p.cols);
        float f[V];
        load_params<T, V>(p.gamma, p.param_f32, e0, lo, hi, vec, 1.f, f);
        g.set(f);
        load_params<T, V>(p.beta, p.param_f32, e0, lo, hi, vec, 0.f, f);
        b.set(f);
    };
    if (EARLY && s0 < s1) params(s0 * V - shift);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (s0 + j * p.tpr < s1) {                     // elements outside the row are zero
            Values<T, V> f;
            f.widen(raw[j]);
            sum += f.sum();
        }
    }
    // Elements of this block's share of the row, their mean, and their squares
    // about it; a cluster joins its shares from these three.
    const int from = max(0, rank * p.per_block * V - shift), to = min(p.cols, (rank + 1) * p.per_block * V - shift);
    const float count = (float)max(0, to - from);
    float mean = row_sum(sum, p.tpr, red[0]) * (p.cs > 1 ? (count > 0.f ? 1.0f / count : 0.f) : p.inv_cols);
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = s0 + j * p.tpr, e0 = s * V - shift;
        if (s < s1) {
            Values<T, V> f;
            f.widen(raw[j]);
            f.minus(mean);
            if (CUT == ENDS && !slot_whole<V>(e0, p.cols)) f.keep(slot_first<CUT>(e0), slot_last<CUT, V>(e0, p.cols));
            sq += f.squares();
        }
    }
    sq = row_sum(sq, p.tpr, red[1]);
    if (p.cs > 1) {
        // sum n_i (m_i - m)^2 + sum s_i: the squares about the row's mean m.
        cg::cluster_group cl_g = cg::this_cluster();
        if (threadIdx.x == 0) share = make_float4(mean, sq, count, 0.f);
        cl_g.sync();
        const int lane = threadIdx.x & 31;
        const float4 o = lane < p.cs ? *cl_g.map_shared_rank(&share, lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        mean = lane_sum(o.x * o.z, 32) * p.inv_cols;
        sq = lane_sum(o.z > 0.f ? o.y + o.z * (o.x - mean) * (o.x - mean) : 0.f, 32);
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");     // (waited for before the block leaves)
    }
    const float rstd = rsqrtf(sq * p.inv_cols + p.eps);
    if (live && t == 0 && rank == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = s0 + j * p.tpr, e0 = s * V - shift;
        if (s < s1) {
            if (!EARLY) params(e0);
            Values<T, V> f;
            f.widen(raw[j]);
            f.minus(mean);
            store_part<T, V>(y + e0, f.affine(rstd, g, b), slot_first<CUT>(e0), slot_last<CUT, V>(e0, p.cols));
        }
    }
    // No block leaves while another may still read its share.
    if (p.cs > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Rows beyond a cluster's registers: the same three steps, re-reading x.
template <typename T, int CUT>
__global__ void __launch_bounds__(1024) layernorm_fwd_long_kernel(const LnParams p) {
    constexpr int V = vec_of<T, CUT>();
    __shared__ float red[2][32];
    __shared__ float cl[2];
    pdl_wait();
    cg::cluster_group cl_g = cg::this_cluster();
    const int rank = (int)(blockIdx.x % p.cs), lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x / p.cs;
    const T* x = static_cast<const T*>(p.x) + row * p.xs;
    T* y = static_cast<T*>(p.y) + row * p.ys;
    const int shift = CUT != ENDS ? 0 : (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int slots = (int)(((int64_t)p.cols + shift + V - 1) / V);
    const int64_t s0 = (int64_t)rank * p.per_block;
    const int64_t s1 = min((int64_t)slots, s0 + p.per_block);
    const bool vec = p.vec_params && shift == 0;
    float sum = 0.f;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
        const int64_t e0 = s * V - shift;
        float f[V];
        widen(load_part<T, V>(x + e0, slot_first<CUT>(e0), slot_last<CUT, V>(e0, p.cols)), f);
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) u += f[i];
        sum += u;
    }
    float mean = row_sum(sum, p.tpr, red[0]);
    if (threadIdx.x == 0) cl[0] = mean;
    cl_g.sync();
    mean = lane_sum(lane < p.cs ? *cl_g.map_shared_rank(&cl[0], lane) : 0.f, 32) * p.inv_cols;
    float sq = 0.f;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
        const int64_t e0 = s * V - shift;
        const int lo = slot_first<CUT>(e0), hi = slot_last<CUT, V>(e0, p.cols);
        float f[V];
        widen(load_part<T, V>(x + e0, lo, hi), f);
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float c = f[i] - mean;
            if (i >= lo && i < hi) u += c * c;
        }
        sq += u;
    }
    sq = row_sum(sq, p.tpr, red[1]);
    if (threadIdx.x == 0) cl[1] = sq;
    cl_g.sync();
    sq = lane_sum(lane < p.cs ? *cl_g.map_shared_rank(&cl[1], lane) : 0.f, 32);
    cl_g.sync();
    const float rstd = rsqrtf(sq * p.inv_cols + p.eps);
    if (threadIdx.x == 0 && rank == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
        const int64_t e0 = s * V - shift;
        const int lo = slot_first<CUT>(e0), hi = slot_last<CUT, V>(e0, p.cols);
        float f[V], g[V], b[V];
        widen(load_part<T, V>(x + e0, lo, hi), f);
        load_params<T, V>(p.gamma, p.param_f32, e0, lo, hi, vec, 1.f, g);
        load_params<T, V>(p.beta, p.param_f32, e0, lo, hi, vec, 0.f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd * g[i] + b[i];
        store_part<T, V>(y + e0, narrow<T, V>(f), lo, hi);
    }
}

// Backward of rows that a block's registers hold.  Group k of the grid takes
// rows k, k + groups, ...; groups is a multiple of the vector length when rows
// start off the 16-byte boundary, so that all rows of a group are cut alike
// and a thread's registers keep the same columns.  Eight elements of a row per
// thread: sums, gamma and two rows in flight fit 64 registers, so 32 warps an
// SM keep the memory busy; a group meets at a barrier of its own.  Short rows
// leave it bound by latency: 65536 x 64 bf16 8.2 us for dx (3.1 TB/s); 1537 x 771
// fp32 in a 776-wide buffer, element by element, 12.5 us.
template <typename T, int CUT, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) layernorm_bwd_kernel(const LnParams p) {
    constexpr int V = vec_of<T, CUT>();
    __shared__ float2 red[2][32];
    extern __shared__ float acc_s[];                   // [group][2][cols] when several groups share the block
    pdl_wait();
    pdl_launch_dependents();                           // one wave: the reduction's blocks wait beside it
    const int tpr = p.tpr, rpb = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x * rpb + sub;
    const T* x0 = static_cast<const T*>(p.x);
    const T* d0 = static_cast<const T*>(p.dy);
    const int shift =
        CUT != ENDS ? 0 : (int)((reinterpret_cast<uintptr_t>(x0 + (int64_t)group * p.xs) & 15u) / sizeof(T));
    const int slots = (p.cols + shift + V - 1) / V;
    const bool vec = p.vec_params && shift == 0;

    float g[NV][V], dg[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = j * tpr + t, e0 = s * V - shift;
        const bool in = s < slots;
        load_params<T, V>(p.gamma, p.param_f32, e0, in ? slot_first<CUT>(e0) : V, in ? slot_last<CUT, V>(e0, p.cols) : 0, vec && in, 1.f,
                          g[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) dg[j][i] = db[j][i] = 0.f;
    }
    // Every group of the block runs the same number of turns.
    const int rows = (int)p.rows, turns = (int)((p.rows - (int64_t)blockIdx.x * rpb + p.groups - 1) / p.groups);
    Vec<T, V> rx[NV], rd[NV];
    float mu = 0.f, r = 0.f;
    if (group < p.rows) {
        load_row<T, CUT, V, NV>(x0 + (int64_t)group * p.xs, p.cols, shift, t, tpr, slots, rx);
        load_row<T, CUT, V, NV>(d0 + (int64_t)group * p.ys, p.cols, shift, t, tpr, slots, rd);
        mu = p.mean_in[group];
        r = p.rstd_in[group];
    }
    // Number of lanes that hold the warps' sums of a row, a power of two.
    const int wpr = tpr >> 5;
    int width = 1;
    while (width < wpr) width <<= 1;
    int64_t row = group;
    for (int it = 0; it < turns; ++it, row += p.groups) {
        const int64_t next = row + p.groups;
        const bool live = row < rows;
        Vec<T, V> nx[NV], nd[NV];
        float nmu = 0.f, nr = 0.f;
        if (next < rows) {                             // under this row's arithmetic
            load_row<T, CUT, V, NV>(x0 + next * p.xs, p.cols, shift, t, tpr, slots, nx);
            load_row<T, CUT, V, NV>(d0 + next * p.ys, p.cols, shift, t, tpr, slots, nd);
            nmu = p.mean_in[next];
            nr = p.rstd_in[next];
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int s = j * tpr + t;
            if (live && s < slots) {
                float fx[V], fd[V];
                widen(rx[j], fx);
                widen(rd[j], fd);
#pragma unroll
                for (int i = 0; i < V; ++i) {          // outside the row dy, and so every term, is zero
                    const float z = (fx[i] - mu) * r, a = fd[i] * g[j][i];
                    s1 += a;
                    s2 += a * z;
                    dg[j][i] += fd[i] * z;
                    db[j][i] += fd[i];
                }
            }
        }
        if (p.dx) {
            s1 = lane_sum(s1, tpr < 32 ? tpr : 32);
            s2 = lane_sum(s2, tpr < 32 ? tpr : 32);
            if (tpr > 32) {
                // Two buffers in turn: a warp that is a row ahead writes the other one.
                float2* buf = red[it & 1];
                if (lane == 0) buf[warp] = make_float2(s1, s2);
                named_bar_sync(1 + sub, tpr);
                const int k = lane & (width - 1);
                const float2 v = k < wpr ? buf[sub * wpr + k] : make_float2(0.f, 0.f);
                s1 = lane_sum(v.x, width);
                s2 = lane_sum(v.y, width);
            }
            s1 *= p.inv_cols;
            s2 *= p.inv_cols;
            if (live) {
                T* dx = static_cast<T*>(p.dx) + row * p.xs;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int s = j * tpr + t, e0 = s * V - shift;
                    if (s < slots) {
                        float fx[V], f[V];
                        widen(rx[j], fx);
                        widen(rd[j], f);
#pragma unroll
                        for (int i = 0; i < V; ++i) f[i] = r * (f[i] * g[j][i] - s1 - (fx[i] - mu) * r * s2);
                        store_part<T, V>(dx + e0, narrow<T, V>(f), slot_first<CUT>(e0), slot_last<CUT, V>(e0, p.cols));
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) { rx[j] = nx[j]; rd[j] = nd[j]; }
        mu = nmu;
        r = nr;
    }
    if (!p.want_params) return;
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
    // Groups that share a warp and its cut are added there first; the rest lie
    // side by side in shared memory and are added in order.
    int held = rpb, mine = sub;
    if (tpr < 32 && p.cut_alike) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                for (int o = tpr; o < 32; o <<= 1) {
                    dg[j][i] += __shfl_xor_sync(0xffffffffu, dg[j][i], o);
                    db[j][i] += __shfl_xor_sync(0xffffffffu, db[j][i], o);
                }
        held = blockDim.x >> 5;
        mine = lane < tpr ? warp : -1;
    }
    float* dst = held > 1 ? acc_s + (int64_t)mine * 2 * p.cols : out;
    if (mine >= 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int s = j * tpr + t, e0 = s * V - shift;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = e0 + i;
                if (s < slots && (CUT != ENDS || (c >= 0 && c < p.cols))) {
                    dst[c] = dg[j][i];
                    dst[p.cols + c] = db[j][i];
                }
            }
        }
    }
    if (held == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.cols; c += blockDim.x) {
        float u = acc_s[c];
        for (int k = 1; k < held; ++k) u += acc_s[k * 2 * p.cols + c];
        out[c] = u;
    }
}

// The same for whole 16-byte aligned rows of at least kBulkBytes, which bulk
// copies bring into a ring in shared memory: the reach of the loads no longer
// depends on registers, and x and dy are read from shared memory twice (sums,
// then dx) instead of being kept.  What bounds this kernel is instructions (46
// an element with eight elements a thread and one row a turn), so a thread
// takes sixteen elements, a turn ROWS rows whose sums share their exchanges and
// barrier, the arithmetic is packed two by two, and rows that fill their threads
// exactly (FULL) get a kernel without the tests for the ones that do not.
// 16384 x 2048 bf16: 32.0 us (6.3 TB/s) for dx, dgamma's parts included; 4096 x
// 8192 32.8 us; 16384 x 1024 fp16 18.0 us (5.6 TB/s).
constexpr int kBulkBytes = 1024, kBulkThreads = 512, kBulkElems = 16, kRingBytes = 192 * 1024, kRingMost = 8;

// The group's sums from its warps' (buf[k][warp], written by the first lane of
// each lane group): sum k in lanes k 32 / N on.
template <int N> __device__ __forceinline__ float group_sums(const float (*buf)[16], int first, int warps) {
    constexpr int kSpan = 32 / N;
    const int lane = threadIdx.x & 31;
    float w = 0.f;
    for (int i = lane % kSpan; i < warps; i += kSpan) w += buf[lane / kSpan][first + i];
#pragma unroll
    for (int d = kSpan / 2; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    return w;
}

template <typename T, int ROWS, bool FULL>
__global__ void __launch_bounds__(kBulkThreads, 1) layernorm_bwd_bulk_kernel(const LnParams p, const int ring_rows) {
    constexpr int V = vec_of<T, WHOLE>(), NV = kBulkElems / V, H = Pairs<T>::N;
    __shared__ float red[2][2 * ROWS][16];
    __shared__ uint64_t bars[8][kRingMost];                // a group is at least two warps
    __shared__ int abort_word;
    extern __shared__ __align__(128) uint8_t ring_s[];     // [group][ring_rows][x row, dy row]; then sums
    volatile int* abort_flag = &abort_word;
    const int tpr = p.tpr, rpb = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x * rpb + sub;
    const uint32_t row_bytes = (uint32_t)p.cols * sizeof(T);
    if (t == 0)
        for (int i = 0; i < ring_rows; ++i) mbar_init(smem_addr(&bars[sub][i]), 1);
    if (threadIdx.x == 0) abort_word = 0;
    mbar_fence_init();
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();                               // one wave: the reduction's blocks wait beside it
    uint8_t* ring = ring_s + (size_t)sub * ring_rows * 2 * row_bytes;
    const int slots = p.cols / V;

    f32x2 g[NV][H], dg[NV][H], db[NV][H];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = j * tpr + t;
        const bool in = FULL || s < slots;
        float f[V];
        load_params<T, V>(p.gamma, p.param_f32, s * V, 0, in ? V : 0, p.vec_params && in, 1.f, f);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            g[j][i] = pack2f(f[2 * i], f[2 * i + 1]);
            dg[j][i] = db[j][i] = 0ull;
        }
    }
    const int mine = group < p.rows ? (int)((p.rows - group + p.groups - 1) / p.groups) : 0;   // this group's rows
    const uint32_t bar0 = smem_addr(&bars[sub][0]), ring0 = smem_addr(ring);
    const int64_t x_step = (int64_t)p.groups * p.xs, d_step = (int64_t)p.groups * p.ys;
    const T* x_next = static_cast<const T*>(p.x) + (int64_t)group * p.xs;
    const T* d_next = static_cast<const T*>(p.dy) + (int64_t)group * p.ys;
    auto issue = [&](int slot) {                           // the next row into its slot (thread 0 of the group)
        const uint32_t bar = bar0 + slot * 8, dst = ring0 + (uint32_t)slot * 2 * row_bytes;
        mbar_arrive_expect_tx(bar, 2 * row_bytes);
        bulk_load(dst, x_next, row_bytes, bar);
        bulk_load(dst + row_bytes, d_next, row_bytes, bar);
        x_next += x_step;
        d_next += d_step;
    };
    int issued = 0;
    if (t == 0)
        for (; issued < ring_rows - ROWS && issued < mine; ++issued) issue(issued);
    const int wpr = tpr >> 5;                              // 2 to 16
    int slot = 0, fill = ring_rows - ROWS;                 // the slots to read and to fill next
    uint32_t phase = 0;
    float mu[ROWS], r[ROWS];
    const float *mean = p.mean_in + group, *rstd = p.rstd_in + group;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        mu[q] = q < mine ? mean[(int64_t)q * p.groups] : 0.f;
        r[q] = q < mine ? rstd[(int64_t)q * p.groups] : 0.f;
    }
    T* dx = static_cast<T*>(p.dx) + (p.dx ? (int64_t)group * p.xs + t * V : 0);
    bool ok = true;
    for (int it = 0, turn = 0; it < mine; it += ROWS, ++turn) {
        float nmu[ROWS], nr[ROWS];
        const uint8_t* src[ROWS];
        f32x2 s1[ROWS], s2[ROWS];
        bool landed = true;
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int64_t at = (int64_t)(it + ROWS + q) * p.groups;
            nmu[q] = it + ROWS + q < mine ? mean[at] : 0.f;
            nr[q] = it + ROWS + q < mine ? rstd[at] : 0.f;
            s1[q] = s2[q] = 0ull;
            src[q] = ring + (size_t)(slot + q) * 2 * row_bytes + t * 16;
            if (it + q < mine) {
                const uint32_t bar = bar0 + (slot + q) * 8;
                const bool here = mbar_try_wait(bar, phase) || mbar_wait(bar, phase, abort_flag);
                landed = landed && here;
                if (here) {
                    const f32x2 nmean = both(-mu[q]), rr = both(r[q]);
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (FULL || j * tpr + t < slots) {
                            f32x2 fx[H], fd[H];
                            Pairs<T>::widen(*reinterpret_cast<const uint4*>(src[q] + j * tpr * 16), fx);
                            Pairs<T>::widen(*reinterpret_cast<const uint4*>(src[q] + row_bytes + j * tpr * 16), fd);
#pragma unroll
                            for (int i = 0; i < H; ++i) {  // with u = dy (x - mean): a z = gamma u r, dy z = u r
                                const f32x2 u = mul2(fd[i], add2(fx[i], nmean));
                                s1[q] = fma2(fd[i], g[j][i], s1[q]);
                                s2[q] = fma2(u, g[j][i], s2[q]);
                                dg[j][i] = fma2(u, rr, dg[j][i]);
                                db[j][i] = add2(db[j][i], fd[i]);
                            }
                        }
                    }
                }
            }
        }
        float v[2 * ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) { v[2 * q] = sum_halves(s1[q]); v[2 * q + 1] = sum_halves(s2[q]); }
        constexpr int kSpan = 32 / (2 * ROWS);             // lanes per sum
        const float part = warp_sums<2 * ROWS>(v);
        float(*buf)[16] = red[turn & 1];                   // two buffers in turn: one barrier a turn is enough
        if (lane % kSpan == 0) buf[lane / kSpan][warp] = part;
        // The group meets once a turn: the sums are there, a wait that ran out
        // stops all of the group, and the previous turn's slots are free.
        ok = named_bar_and(1 + sub, tpr, landed);
        if (!ok) break;
        if (t == 0)
            for (int q = 0; q < ROWS && issued < mine; ++q, ++issued) issue(fill + q);
        fill = fill + ROWS == ring_rows ? 0 : fill + ROWS;
        slot += ROWS;
        if (slot == ring_rows) { slot = 0; phase ^= 1; }
        if (p.dx) {
            const float w = group_sums<2 * ROWS>(buf, sub * wpr, wpr) * p.inv_cols;
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                const float t1 = __shfl_sync(0xffffffffu, w, 2 * q * kSpan) * r[q];
                const float t2 = __shfl_sync(0xffffffffu, w, (2 * q + 1) * kSpan) * r[q] * r[q] * r[q];
                if (it + q < mine) {
                    // dx = r a - r mean(a) - (x - mean) r^3 mean(gamma u)
                    const f32x2 nmean = both(-mu[q]), rr = both(r[q]), n1 = both(-t1), n2 = both(-t2);
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (FULL || j * tpr + t < slots) {
                            f32x2 fx[H], fd[H];
                            Pairs<T>::widen(*reinterpret_cast<const uint4*>(src[q] + j * tpr * 16), fx);
                            Pairs<T>::widen(*reinterpret_cast<const uint4*>(src[q] + row_bytes + j * tpr * 16), fd);
#pragma unroll
                            for (int i = 0; i < H; ++i)
                                fd[i] = fma2(mul2(fd[i], g[j][i]), rr, fma2(add2(fx[i], nmean), n2, n1));
                            *reinterpret_cast<uint4*>(dx + j * tpr * V) = Pairs<T>::narrow(fd);
                        }
                    }
                    dx += x_step;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) { mu[q] = nmu[q]; r[q] = nr[q]; }
    }
    // Copies still in flight after a wait that ran out land before the block leaves.
    if (t == 0 && !ok)
        for (int i = issued > ring_rows ? issued - ring_rows : 0; i < issued; ++i)
            mbar_drain_wait(bar0 + (i % ring_rows) * 8, (uint32_t)(i / ring_rows) & 1u);
    if (!p.want_params) return;
    // The groups' sums side by side where the ring was, then added in order.
    float4* acc_s = reinterpret_cast<float4*>(ring_s);     // [group][2][cols]
    const int quads = p.cols / 4;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (FULL || j * tpr + t < slots) {
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const int at = sub * 2 * quads + ((j * tpr + t) * V + 2 * i) / 4;
                float4 u, w;
                unpack2f(dg[j][i], u.x, u.y);
                unpack2f(dg[j][i + 1], u.z, u.w);
                unpack2f(db[j][i], w.x, w.y);
                unpack2f(db[j][i + 1], w.z, w.w);
                acc_s[at] = u;
                acc_s[at + quads] = w;
            }
        }
    }
    __syncthreads();
    float4* out = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * 2 * p.cols);
    for (int c = threadIdx.x; c < 2 * quads; c += blockDim.x) {
        float4 u = acc_s[c];
        for (int k = 1; k < rpb; ++k) {
            const float4 w = acc_s[k * 2 * quads + c];
            u.x += w.x; u.y += w.y; u.z += w.z; u.w += w.w;
        }
        out[c] = u;
    }
}

// Forward of the same rows: a turn's rows go from the ring into registers, so
// their slots are free again after the turn's one meeting: each warp takes the
// squares about the mean of its own share, and the shares are joined exactly
// (a second meeting for the squares cost 2 to 4 us more).  16384 x 2048 bf16 28.9
// us (4.6 TB/s), 4096 x 8192 29.0, 8192 x 4096 fp32 46.2 (5.8 TB/s), 16384 x 1024
// fp16 15.5; 16384 x 2040 fp16, whose rows do not fill their threads, 37.2.
template <typename T, int ROWS, bool FULL>
__global__ void __launch_bounds__(kBulkThreads, 1) layernorm_fwd_bulk_kernel(const LnParams p, const int ring_rows) {
    constexpr int V = vec_of<T, WHOLE>(), NV = kBulkElems / V, H = Pairs<T>::N, kSpan = 32 / ROWS;
    constexpr int kLook = kSpan < 16 ? 16 / kSpan : 1;     // warps of a group (16 at most) that a lane joins
    __shared__ float2 red[2][ROWS][16];                    // (mean, squares about it) of each warp's share
    __shared__ uint64_t bars[8][kRingMost];
    __shared__ int abort_word;
    extern __shared__ __align__(128) uint8_t ring_s[];     // [group][ring_rows][row]
    volatile int* abort_flag = &abort_word;
    const int tpr = p.tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpb = blockDim.x / tpr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wpr = tpr >> 5;
    const int group = blockIdx.x * rpb + sub;
    const uint32_t row_bytes = (uint32_t)p.cols * sizeof(T);
    if (t == 0)
        for (int i = 0; i < ring_rows; ++i) mbar_init(smem_addr(&bars[sub][i]), 1);
    if (threadIdx.x == 0) abort_word = 0;
    mbar_fence_init();
    __syncthreads();
    pdl_wait();
    const uint8_t* ring = ring_s + (size_t)sub * ring_rows * row_bytes;
    const uint32_t bar0 = smem_addr(&bars[sub][0]), ring0 = smem_addr(ring);
    const int slots = p.cols / V;
    const int mine = group < p.rows ? (int)((p.rows - group + p.groups - 1) / p.groups) : 0;   // this group's rows
    const int64_t x_step = (int64_t)p.groups * p.xs, y_step = (int64_t)p.groups * p.ys;
    const T* x_next = static_cast<const T*>(p.x) + (int64_t)group * p.xs;
    T* y = static_cast<T*>(p.y) + (int64_t)group * p.ys + t * V;
    auto issue = [&](int slot) {                           // the next row into its slot (thread 0 of the group)
        mbar_arrive_expect_tx(bar0 + slot * 8, row_bytes);
        bulk_load(ring0 + (uint32_t)slot * row_bytes, x_next, row_bytes, bar0 + slot * 8);
        x_next += x_step;
    };
    int issued = 0;
    if (t == 0)
        for (; issued < ring_rows && issued < mine; ++issued) issue(issued);
    f32x2 g[NV][H], b[NV][H];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int s = j * tpr + t;
        const bool in = FULL || s < slots;
        float f[V], h[V];
        load_params<T, V>(p.gamma, p.param_f32, s * V, 0, in ? V : 0, p.vec_params && in, 1.f, f);
        load_params<T, V>(p.beta, p.param_f32, s * V, 0, in ? V : 0, p.vec_params && in, 0.f, h);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            g[j][i] = pack2f(f[2 * i], f[2 * i + 1]);
            b[j][i] = pack2f(h[2 * i], h[2 * i + 1]);
        }
    }
    // Elements of a warp's share of a row, and one over this warp's.
    auto share_of = [&](int w) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) n += min(32, max(0, slots - j * tpr - w * 32));
        return (float)(n * V);
    };
    const float own = share_of(warp - sub * wpr), inv_own = own > 0.f ? 1.0f / own : 0.f;
    float size[kLook];
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
        const int w = lane % kSpan + k * kSpan;
        size[k] = w < wpr ? share_of(w) : 0.f;
    }
    int slot = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = 0; it < mine; it += ROWS) {
        f32x2 f[ROWS][NV][H];
        float v[ROWS];
        bool landed = true;
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            f32x2 s = 0ull;
            if (it + q < mine) {
                const uint32_t bar = bar0 + (slot + q) * 8;
                const bool here = mbar_try_wait(bar, phase) || mbar_wait(bar, phase, abort_flag);
                landed = landed && here;
                if (here) {
                    const uint8_t* src = ring + (size_t)(slot + q) * row_bytes + t * 16;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (FULL || j * tpr + t < slots) {
                            Pairs<T>::widen(*reinterpret_cast<const uint4*>(src + j * tpr * 16), f[q][j]);
#pragma unroll
                            for (int i = 0; i < H; ++i) s = add2(s, f[q][j][i]);
                        }
                    }
                }
            }
            v[q] = sum_halves(s);
        }
        const float warp_mean = warp_sums<ROWS>(v) * inv_own;
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const f32x2 m = both(-__shfl_sync(0xffffffffu, warp_mean, q * kSpan));
            f32x2 s = 0ull;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (FULL || j * tpr + t < slots) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const f32x2 d = add2(f[q][j][i], m);
                        s = fma2(d, d, s);
                    }
                }
            }
            v[q] = sum_halves(s);
        }
        const float warp_sq = warp_sums<ROWS>(v);
        if (lane % kSpan == 0) red[turn][lane / kSpan][warp] = make_float2(warp_mean, warp_sq);
        ok = named_bar_and(1 + sub, tpr, landed);
        if (!ok) break;
        if (t == 0)
            for (int q = 0; q < ROWS && issued < mine; ++q, ++issued) issue(slot + q);
        slot += ROWS;
        if (slot == ring_rows) { slot = 0; phase ^= 1; }
        // The row's mean m, and sum s_i + n_i (m_i - m)^2: the squares about it.
        float2 o[kLook];
        float total = 0.f, sq = 0.f;
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            const int w = lane % kSpan + k * kSpan;
            o[k] = w < wpr ? red[turn][lane / kSpan][sub * wpr + w] : make_float2(0.f, 0.f);
            total = fmaf(o[k].x, size[k], total);
        }
        turn ^= 1;                                         // (the other half is free: all have met since it was read)
        total = lane_sum(total, kSpan) * p.inv_cols;
#pragma unroll
        for (int k = 0; k < kLook; ++k) sq += fmaf(size[k] * (o[k].x - total), o[k].x - total, o[k].y);
        sq = lane_sum(sq, kSpan) * p.inv_cols;
        float mean[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            mean[q] = __shfl_sync(0xffffffffu, total, q * kSpan);
            const f32x2 m = both(-mean[q]);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (FULL || j * tpr + t < slots)
#pragma unroll
                    for (int i = 0; i < H; ++i) f[q][j][i] = add2(f[q][j][i], m);
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const float rstd = rsqrtf(__shfl_sync(0xffffffffu, sq, q * kSpan) + p.eps);
            if (it + q < mine) {
                if (t == 0) {
                    const int64_t row = group + (int64_t)(it + q) * p.groups;
                    if (p.mean) p.mean[row] = mean[q];
                    if (p.rstd) p.rstd[row] = rstd;
                }
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (FULL || j * tpr + t < slots) {
                        f32x2 o[H];
#pragma unroll
                        for (int i = 0; i < H; ++i) o[i] = fma2(mul2(f[q][j][i], both(rstd)), g[j][i], b[j][i]);
                        *reinterpret_cast<uint4*>(y + j * tpr * V) = Pairs<T>::narrow(o);
                    }
                }
                y += y_step;
            }
        }
    }
    // Copies still in flight after a wait that ran out land before the block leaves.
    if (t == 0 && !ok)
        for (int i = issued > ring_rows ? issued - ring_rows : 0; i < issued; ++i)
            mbar_drain_wait(bar0 + (i % ring_rows) * 8, (uint32_t)(i / ring_rows) & 1u);
}

// Long rows, pass 1 (both passes of 31 x 99999 fp16 take 12.3 us, of 32 x
// 200704 21 us; their dgamma and dbeta as much again): sum a and sum a z of one row's share of columns.
template <typename T, int CUT>
__global__ void __launch_bounds__(256) layernorm_bwd_sums_kernel(const LnParams p, float2* sums) {
    constexpr int V = vec_of<T, CUT>();
    __shared__ float red[2][32];
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.xs;
    const T* dy = static_cast<const T*>(p.dy) + row * p.ys;
    const int shift = CUT != ENDS ? 0 : (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int64_t slots = ((int64_t)p.cols + shift + V - 1) / V;
    const int64_t per = (slots + gridDim.y - 1) / gridDim.y;
    const int64_t s0 = blockIdx.y * per, s1 = min(slots, s0 + per);
    const bool vec = p.vec_params && shift == 0;
    const float mu = p.mean_in[row], r = p.rstd_in[row];
    float a1 = 0.f, a2 = 0.f;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
        const int64_t e0 = s * V - shift;
        const int lo = slot_first<CUT>(e0), hi = slot_last<CUT, V>(e0, p.cols);
        float fx[V], fd[V], g[V];
        widen(load_part<T, V>(x + e0, lo, hi), fx);
        widen(load_part<T, V>(dy + e0, lo, hi), fd);
        load_params<T, V>(p.gamma, p.param_f32, e0, lo, hi, vec, 1.f, g);
        float u1 = 0.f, u2 = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= lo && i < hi) {
                const float a = fd[i] * g[i];
                u1 += a;
                u2 += a * ((fx[i] - mu) * r);
            }
        }
        a1 += u1;
        a2 += u2;
    }
    a1 = row_sum(a1, blockDim.x, red[0]);
    a2 = row_sum(a2, blockDim.x, red[1]);
    if (threadIdx.x == 0) sums[row * gridDim.y + blockIdx.y] = make_float2(a1, a2);
}

// Long rows, pass 2: a thread owns one vector of columns and runs down every
// gridDim.y-th row (a multiple of the vector length when rows are cut
// differently, as above), writing dx and adding dgamma and dbeta.
template <typename T, int CUT>
__global__ void __launch_bounds__(128) layernorm_bwd_cols_kernel(const LnParams p, const float2* sums, int shares) {
    constexpr int V = vec_of<T, CUT>();
    pdl_wait();
    const T* x0 = static_cast<const T*>(p.x) + (int64_t)blockIdx.y * p.xs;
    const int shift = CUT != ENDS ? 0 : (int)((reinterpret_cast<uintptr_t>(x0) & 15u) / sizeof(T));
    const int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, e0 = s * V - shift;
    if (e0 >= p.cols) return;
    const int lo = slot_first<CUT>(e0), hi = slot_last<CUT, V>(e0, p.cols);
    const bool vec = p.vec_params && shift == 0;
    float g[V], dg[V], db[V];
    load_params<T, V>(p.gamma, p.param_f32, e0, lo, hi, vec, 1.f, g);
#pragma unroll
    for (int i = 0; i < V; ++i) dg[i] = db[i] = 0.f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        float s1 = 0.f, s2 = 0.f;
        for (int k = 0; k < shares; ++k) {
            const float2 u = sums[row * shares + k];
            s1 += u.x;
            s2 += u.y;
        }
        s1 *= p.inv_cols;
        s2 *= p.inv_cols;
        const float mu = p.mean_in[row], r = p.rstd_in[row];
        float fx[V], fd[V], f[V];
        widen(load_part<T, V>(static_cast<const T*>(p.x) + row * p.xs + e0, lo, hi), fx);
        widen(load_part<T, V>(static_cast<const T*>(p.dy) + row * p.ys + e0, lo, hi), fd);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = (fx[i] - mu) * r;
            f[i] = r * (fd[i] * g[i] - s1 - z * s2);
            dg[i] += fd[i] * z;                        // (outside the row nothing is stored)
            db[i] += fd[i];
        }
        if (p.dx)
            store_part<T, V>(static_cast<T*>(p.dx) + row * p.xs + e0, narrow<T, V>(f), lo, hi);
    }
    if (!p.want_params) return;
    float* out = p.part + (int64_t)blockIdx.y * 2 * p.cols + e0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= lo && i < hi) {
            out[i] = dg[i];
            out[p.cols + i] = db[i];
        }
    }
}

// dgamma and dbeta: the parts' columns added in order, SPAN columns by 1024 /
// SPAN shares of the parts per block (blockIdx.y: dgamma or dbeta).  A few
// hundred parts of a normal row: 32 shares, about ten loads per thread, all in
// flight.  A few parts of a long row: one share.  One trip to memory and the
// launch are the whole of its 3 to 5 us.
template <int SPAN>
__global__ void __launch_bounds__(1024) layernorm_params_kernel(const float* part, int parts, int cols, void* dgamma,
                                                                void* dbeta, int f32, int bf16) {
    constexpr int SHARES = 1024 / SPAN;
    pdl_wait();
    void* out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    const int at = threadIdx.x % SPAN, k = threadIdx.x / SPAN;
    const int64_t c = (int64_t)blockIdx.x * SPAN + at;
    float v = 0.f;
    if (c < cols) {
        const float* q = part + (int64_t)blockIdx.y * cols + c;
        const int64_t pitch = 2 * (int64_t)cols;
#pragma unroll 10
        for (int i = k; i < parts; i += SHARES) v += q[i * pitch];
    }
    if constexpr (SHARES == 1) {
        if (c < cols) store_param(out, f32, bf16, c, v);
    } else {
        static_assert(SPAN == 32, "a warp per column");
        __shared__ float sh[32][33];
        sh[k][at] = v;
        __syncthreads();
        v = lane_sum(sh[at][k], 32);                   // warp k adds column k's shares
        const int64_t col = (int64_t)blockIdx.x * 32 + k;
        if (at == 0 && col < cols) store_param(out, f32, bf16, col, v);
    }
}

// ------------------------------------------------------------------ host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads for `slots` vectors of a row at nv vectors per thread: a power of
// two below a warp, else whole warps.
int threads_for(int64_t slots, int nv) {
    const int64_t t = ceil_div(slots, nv);
    if (t >= 32) return (int)(ceil_div(t, 32) * 32);
    int p = 1;
    while (p < t) p <<= 1;
    return p;
}

constexpr int kBwdElems = 8;          // backward: elements of a row per thread at most (registers)
constexpr int kBwdCols = kBwdElems * 1024;

// Blocks of the in-block form at most: 1024 threads an SM, in blocks of 512 or
// one of 1024; rounded up to whole vectors of groups.
int bwd_grid(int tpr) { return device_sm_count() * (tpr > 512 ? 1 : 2); }

// Blocks per row of the long form's sums at most: eight blocks per SM in all.
int64_t long_shares(int64_t rows) {
    const int64_t s = rows ? ceil_div(8 * device_sm_count(), rows) : 1;
    return s > 64 ? 64 : s;
}

// Whether a call's tensors can move in 16-byte vectors: every row of all of
// them sits alike against the 16-byte boundary.
bool same_phase(const void* a, int64_t sa, const void* b, int64_t sb, size_t e) {
    return (reinterpret_cast<uintptr_t>(a) & 15) == (reinterpret_cast<uintptr_t>(b) & 15) &&
           ((sa - sb) * (int64_t)e) % 16 == 0;
}

// The cut of a call that moves vectors.
int cut_of(const void* x, int64_t xs, int64_t cols, size_t e) {
    const bool whole = aligned_to(x, 16) && xs * (int64_t)e % 16 == 0 && cols * (int64_t)e % 16 == 0;
    return whole ? WHOLE : ENDS;
}

// The ring of a bulk kernel of `rows_held` rows per slot (x; or x and dy): two
// rows a turn where the ring then still holds two on their way.  False when the
// call is not for it: rows that are cut or short, or fewer than two a group
// (there would be nothing to run ahead of).
struct BulkPlan { int tpr, rpb, rows; bool twice, full; size_t smem; };
bool bulk_plan(const LnParams& p, int cut, size_t e, int rows_held, BulkPlan* b) {
    const int64_t row_bytes = p.cols * (int64_t)e, slots = row_bytes / 16;
    if (cut != WHOLE || row_bytes < kBulkBytes || p.cols > kBwdCols) return false;
    b->tpr = threads_for(slots, kBulkElems * (int)e / 16);
    if (b->tpr < 64) b->tpr = 64;
    b->full = (int64_t)b->tpr * (kBulkElems * (int)e / 16) == slots;
    b->rpb = kBulkThreads / b->tpr;
    if (p.rows < 2 * (int64_t)device_sm_count() * b->rpb) return false;
    b->rows = (int)(kRingBytes / (b->rpb * rows_held * row_bytes));
    if (b->rows > kRingMost) b->rows = kRingMost;
    b->twice = b->rows >= 4;
    if (b->twice) b->rows &= ~1;
    b->smem = (size_t)b->rpb * b->rows * rows_held * row_bytes;
    return true;
}

template <typename T> cudaError_t fwd_typed(const layernorm_desc& d, LnParams p, cudaStream_t st) {
    const bool scalar = !same_phase(p.x, p.xs, p.y, p.ys, sizeof(T));
    const int cut = scalar ? SINGLE : cut_of(p.x, p.xs, p.cols, sizeof(T));
    const int V = scalar ? 1 : 16 / (int)sizeof(T);
    BulkPlan bulk;
    if (p.cols * (int64_t)sizeof(T) >= 2 * kBulkBytes && bulk_plan(p, cut, sizeof(T), 1, &bulk)) {
        p.tpr = bulk.tpr;
        p.groups = device_sm_count() * bulk.rpb;
#define LN_FWD_BULK(FULL)                                          \
    (bulk.rows == 8 ? layernorm_fwd_bulk_kernel<T, 4, FULL>        \
     : bulk.twice   ? layernorm_fwd_bulk_kernel<T, 2, FULL>        \
                    : layernorm_fwd_bulk_kernel<T, 1, FULL>)
        auto kern = bulk.full ? LN_FWD_BULK(true) : LN_FWD_BULK(false);
#undef LN_FWD_BULK
        const cudaError_t e = allow_smem(kern, kRingBytes);
        if (e != cudaSuccess) return e;
        return launch_after(kern, dim3((unsigned)device_sm_count()), dim3(bulk.rpb * bulk.tpr), bulk.smem, st, p,
                            bulk.rows);
    }
    // Vectors of the most unevenly cut row.
    const int shift = scalar                                  ? 0
                      : (p.xs * (int64_t)sizeof(T)) % 16 == 0 ? (int)((reinterpret_cast<uintptr_t>(p.x) & 15u) / sizeof(T))
                                                              : V - 1;
    const int64_t slots = ceil_div((int64_t)p.cols + shift, V);
    // Vectors per thread: as few as keep every row's threads resident at once
    // (64 warps an SM), so that small calls spread over the GPU and large
    // ones keep several loads per thread in flight.
    const int64_t room = (int64_t)device_sm_count() * 2048;
    int nv = 1;
    while (nv < 4 && p.rows * threads_for(slots, nv) > room) nv *= 2;
    while (nv < 8 && threads_for(slots, nv) > 1024) nv *= 2;
    int64_t threads = threads_for(slots, nv), grid;
    bool is_long = false;
    p.cs = 1;
    if (threads > 1024 || (slots >= 2048 && p.rows * 2 <= device_sm_count())) {
        // One row over a cluster: the fewest blocks that hold it, then more
        // while the GPU has SMs to spare and a thread would keep a vector.
        while (p.cs < 8 && (threads_for(ceil_div(slots, p.cs), 8) > 1024 ||
                            (p.rows * p.cs * 2 <= device_sm_count() && ceil_div(slots, p.cs * 2) >= 256)))
            p.cs *= 2;
        p.per_block = (int)ceil_div(slots, p.cs);
        nv = 1;
        while (nv < 8 && threads_for(p.per_block, nv) > (nv < 4 ? 512 : 1024)) nv *= 2;
        threads = threads_for(p.per_block, nv);
        is_long = threads > 1024;
        if (is_long) threads = 1024;
        grid = p.rows * p.cs;
        p.tpr = (int)threads;
    } else {
        p.per_block = (int)slots;
        p.tpr = (int)threads;
        const int64_t rpb = threads >= 256 ? 1 : 256 / threads;
        threads *= rpb;
        grid = ceil_div(p.rows, rpb);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (is_long)
        return cudaLaunchKernelEx(&cfg, cut == SINGLE ? layernorm_fwd_long_kernel<T, SINGLE>
                                        : cut == ENDS ? layernorm_fwd_long_kernel<T, ENDS>
                                                      : layernorm_fwd_long_kernel<T, WHOLE>, p);
#define LN_FWD(NV)                                                              \
    cudaLaunchKernelEx(&cfg, cut == SINGLE ? layernorm_fwd_kernel<T, SINGLE, NV> \
                             : cut == ENDS ? layernorm_fwd_kernel<T, ENDS, NV>   \
                                           : layernorm_fwd_kernel<T, WHOLE, NV>, p)
    switch (nv) {
        case 1: return LN_FWD(1);
        case 2: return LN_FWD(2);
        case 4: return LN_FWD(4);
        default: return LN_FWD(8);
    }
#undef LN_FWD
}

template <typename T> cudaError_t bwd_typed(const layernorm_desc& d, LnParams p, float* ws, int* parts, cudaStream_t st) {
    const bool scalar = !same_phase(p.x, p.xs, p.dy, p.ys, sizeof(T)) ||
                        (p.dx && !same_phase(p.x, p.xs, p.dx, p.xs, sizeof(T)));
    const int cut = scalar ? SINGLE : cut_of(p.x, p.xs, p.cols, sizeof(T));
    const int V = scalar ? 1 : 16 / (int)sizeof(T);
    const bool cut_alike = scalar || (p.xs * (int64_t)sizeof(T)) % 16 == 0;
    const int most_shift = scalar     ? 0
                           : cut_alike ? (int)((reinterpret_cast<uintptr_t>(p.x) & 15u) / sizeof(T))
                                       : V - 1;
    const int64_t slots = ceil_div((int64_t)p.cols + most_shift, V);
    const int sms = device_sm_count();
    p.cut_alike = cut_alike;
    BulkPlan bulk;
    if (bulk_plan(p, cut, sizeof(T), 2, &bulk)) {
        p.tpr = bulk.tpr;
        p.groups = sms * bulk.rpb;
        *parts = sms;
        const size_t sums = (size_t)bulk.rpb * 2 * p.cols * sizeof(float), smem = bulk.smem > sums ? bulk.smem : sums;
        auto kern = bulk.full ? (bulk.twice ? layernorm_bwd_bulk_kernel<T, 2, true> : layernorm_bwd_bulk_kernel<T, 1, true>)
                              : (bulk.twice ? layernorm_bwd_bulk_kernel<T, 2, false>
                                            : layernorm_bwd_bulk_kernel<T, 1, false>);
        const cudaError_t e = allow_smem(kern, kRingBytes);        // (the sums take 64 KB at most)
        if (e != cudaSuccess) return e;
        return launch_after(kern, dim3((unsigned)sms), dim3(bulk.rpb * bulk.tpr), smem, st, p, bulk.rows);
    }
    if (slots * V <= kBwdCols) {
        // As many threads a row as keep one vector each, or eight elements.
        int nv = 1;
        const int64_t room = (int64_t)sms * 1024;
        while (nv * V < kBwdElems && (threads_for(slots, nv) > 1024 || p.rows * threads_for(slots, nv) > room)) nv *= 2;
        p.tpr = threads_for(slots, nv);
        const int block = p.tpr > 512 ? p.tpr : 512 / p.tpr * p.tpr;
        const int rpb = block / p.tpr;
        int64_t grid = ceil_div(p.rows, rpb);
        if (grid > bwd_grid(p.tpr)) grid = bwd_grid(p.tpr);
        if (!cut_alike) grid = ceil_div(grid, V) * V;
        p.groups = (int)grid * rpb;
        *parts = (int)grid;
        const size_t smem = rpb > 1 && p.want_params ? (size_t)rpb * 2 * p.cols * sizeof(float) : 0;   // 32 KB at most
#define LN_BWD_AT(CUT, NV, TH) launch_after(layernorm_bwd_kernel<T, CUT, NV, TH>, dim3((unsigned)grid), dim3(block), smem, st, p)
#define LN_BWD(CUT, NV) (block > 512 ? LN_BWD_AT(CUT, NV, 1024) : LN_BWD_AT(CUT, NV, 512))
        if (cut == SINGLE) {
            switch (nv) {
                case 1: return LN_BWD(SINGLE, 1);
                case 2: return LN_BWD(SINGLE, 2);
                case 4: return LN_BWD(SINGLE, 4);
                default: return LN_BWD(SINGLE, 8);
            }
        }
        if constexpr (sizeof(T) == 4) {
            if (nv == 2) return cut == ENDS ? LN_BWD(ENDS, 2) : LN_BWD(WHOLE, 2);
        }
        return cut == ENDS ? LN_BWD(ENDS, 1) : LN_BWD(WHOLE, 1);
#undef LN_BWD
#undef LN_BWD_AT
    }
    // Two passes: row sums, then columns.  Enough shares of the columns, and
    // of the rows, to fill the GPU.
    int64_t shares = long_shares(p.rows);
    if (shares > ceil_div(slots, 1024)) shares = ceil_div(slots, 1024);
    float2* sums = reinterpret_cast<float2*>(ws);
    cudaError_t e = cudaSuccess;
    if (p.dx) {
        e = launch_after(cut == SINGLE ? layernorm_bwd_sums_kernel<T, SINGLE> : layernorm_bwd_sums_kernel<T, ENDS>,
                         dim3((unsigned)p.rows, (unsigned)shares), dim3(256), 0, st, p, sums);
        if (e != cudaSuccess) return e;
    }
    const int64_t gx = ceil_div(slots, 128);
    int64_t gy = ceil_div(8 * sms, gx);
    if (gy > 64) gy = 64;
    if (gy > p.rows) gy = p.rows;
    if (!cut_alike) gy = ceil_div(gy, V) * V;
    if (gy > 64) gy = 64;
    *parts = (int)gy;
    return launch_after(cut == SINGLE ? layernorm_bwd_cols_kernel<T, SINGLE> : layernorm_bwd_cols_kernel<T, ENDS>,
                        dim3((unsigned)gx, (unsigned)gy), dim3(128), 0, st, p, static_cast<const float2*>(sums),
                        p.dx ? (int)shares : 0);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const layernorm_desc& d, const void* x, const void* gamma, const void* beta, void* y,
                                 float* mean, float* rstd, cudaStream_t st) {
    if (d.pixels) return launch_layernorm_planes_fwd(d, x, gamma, beta, y, mean, rstd, st);
    LnParams p{};
    p.rows = d.rows; p.xs = d.xs; p.ys = d.ys; p.cols = (int)d.cols;
    p.param_f32 = d.param == CONV2D_F32;
    p.vec_params = aligned_to(gamma, 16) && aligned_to(beta, 16);
    p.eps = d.eps;
    p.inv_cols = 1.0f / (float)d.cols;
    p.x = x; p.gamma = gamma; p.beta = beta; p.y = y; p.mean = mean; p.rstd = rstd;
    switch (d.dtype) {
        case CONV2D_F32: return fwd_typed<float>(d, p, st);
        case CONV2D_F16: return fwd_typed<__half>(d, p, st);
        default: return fwd_typed<__nv_bfloat16>(d, p, st);
    }
}

// Row sums of the long form (rows x shares pairs), then the parts of dgamma
// and dbeta (blocks of the in-block form, or row shares of the long one).
// Which form runs depends on the tensors' alignment when a vector more or
// less decides, so the sizes allow for both.
static size_t bwd_sums_bytes(const layernorm_desc& d) {
    if (d.cols <= kBwdCols - 8) return 0;
    return align_up((size_t)(d.rows * long_shares(d.rows)) * sizeof(float2), 256);
}

size_t layernorm_bwd_workspace(const layernorm_desc& d) {
    if (d.pixels) return layernorm_planes_bwd_workspace(d);
    const size_t parts = d.cols <= kBwdCols ? (size_t)bwd_grid(1) + 8 : 64;
    return bwd_sums_bytes(d) + parts * 2 * (size_t)d.cols * sizeof(float);
}

cudaError_t status_word_ln(void** p) { return unit_status_word(p); }
cudaError_t wait_limit_set_ln(cudaStream_t st, uint64_t ns) { return unit_wait_limit_set(st, ns); }

cudaError_t launch_layernorm_params(const float* part, int parts, const layernorm_desc& d, void* dgamma, void* dbeta,
                                    cudaStream_t st) {
    const int span = parts > 64 || d.cols < 1024 ? 32 : 1024;
    return launch_after(span == 32 ? layernorm_params_kernel<32> : layernorm_params_kernel<1024>,
                        dim3((unsigned)((d.cols + span - 1) / span), 2), dim3(1024), 0, st, part, parts, (int)d.cols,
                        dgamma, dbeta, d.param == CONV2D_F32 ? 1 : 0, d.param == CONV2D_BF16 ? 1 : 0);
}

cudaError_t launch_layernorm_bwd(const layernorm_desc& d, const void* dy, const void* x, const void* gamma,
                                 const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* ws,
                                 cudaStream_t st) {
    if (d.pixels) return launch_layernorm_planes_bwd(d, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, st);
    LnParams p{};
    p.rows = d.rows; p.xs = d.xs; p.ys = d.ys; p.cols = (int)d.cols;
    p.param_f32 = d.param == CONV2D_F32;
    p.vec_params = aligned_to(gamma, 16);
    p.inv_cols = 1.0f / (float)d.cols;
    p.x = x; p.dy = dy; p.gamma = gamma; p.dx = dx; p.mean_in = mean; p.rstd_in = rstd;
    p.want_params = dgamma || dbeta;
    float* sums = static_cast<float*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + bwd_sums_bytes(d));
    int parts = 0;
    cudaError_t e;
    switch (d.dtype) {
        case CONV2D_F32: e = bwd_typed<float>(d, p, sums, &parts, st); break;
        case CONV2D_F16: e = bwd_typed<__half>(d, p, sums, &parts, st); break;
        default: e = bwd_typed<__nv_bfloat16>(d, p, sums, &parts, st);
    }
    if (e != cudaSuccess || !p.want_params) return e;
    return launch_layernorm_params(p.part, parts, d, dgamma, dbeta, st);
}

}  // namespace conv2d_gb300
