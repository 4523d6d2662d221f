// Linear cross entropy over a large vocabulary, forward and backward, on the
// 5th-generation tensor cores (tcgen05 MMA, accumulators in tensor memory,
// operands fed by TMA).
//
//   forward    z = h w^T one 128 x BN tile at a time; the epilogue reduces
//              each row of the tile to (max, sum exp(z - max)) and picks the
//              target's z, so z never reaches memory.  A second kernel joins
//              the tiles' pairs: the maximum first, then the rescaled sums.
//   backward   per piece of the vocabulary: z again, turned by the epilogue
//              into dz = g (exp(z - lse) - [v = y]) in 16 bits; then
//              dh += dz w and dw = dz^T h.
//
// All three products run in one kernel (ce_gemm_kernel): C[M][N] = sum_k
// A[m][k] B[n][k] in 64-wide K chunks, each operand stored either along K
// (K-major) or along its own rows (MN-major: dz for dw, w for dh, h for dw),
// so nothing is transposed in memory.  dz is stored without the part of g that
// all rows share (the whole of it for the sum and the mean), which multiplies
// the fp32 result instead: rounding it into every element would shift them all
// the same way.  Per-row factors are scaled so that the largest is just below
// 2^15: fp16's range then reaches down to probabilities of 2^-39 of it.
//
// fp32 operands are split into three bf16 parts each (8 significand bits, 24
// together) and the six products of parts that matter are accumulated, the
// small ones first: the parts are neighbouring column blocks of one packed
// matrix, and the K loop runs six times as long.
//
// The tensor cores round an accumulator toward zero at every step, a bias that
// grows with K (4e-5 of dh over 20011 vocabulary rows, measured).  Where the
// result is kept in fp32 (the losses, and everything of fp32 operands) the
// accumulator therefore runs for `seg` chunks only and the epilogue adds these
// partial sums in registers, rounded to nearest, while the next ones are
// computed (PROMOTE).
//
// Few rows by many columns (or a long K by a small output) is split over K and
// joined by a second kernel in a fixed order, so that all SMs have work.
#include <cuda.h>
#include <math.h>

#include <mutex>
#include <set>
#include <utility>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kBM = 128, kBK = 64;            // MMA rows; K elements per stage (128 bytes)
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxRing = 8;
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kStageWarpBytes = 32 * 17 * 4;  // epilogue staging per warp: 32 rows of 17 words
constexpr int kSmemMost = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f;

enum Epilogue { EPI_LSE = 0, EPI_DZ = 1, EPI_OUT = 2 };

struct GemmParams {
    int M, N;                // valid extents of C
    int BN, n_m, n_n;        // tile width, tiles
    int group;               // row tiles that share each column tile before the next one is taken
    int nk, pairs;           // K chunks of one product of parts, and such products (1 or 6)
    int a_part, b_part;      // column offset from one part to the next
    int splits;
    int stages;
    int seg;                 // PROMOTE: chunks per accumulation in tensor memory
    // EPI_LSE and EPI_DZ
    int col0;                // first vocabulary row of this piece
    int vocab;
    int64_t ignore;
    const int64_t* target;
    float2* lse_part;        // [(column tile, half)][M]
    float* z_target;         // [M]
    const float *lse, *coef; // [M]
    void* dz;                // [M][parts * dz_part]
    int dz_part, parts;
    // EPI_OUT
    void* out;               // final element type, or the fp32 partial sums [split][M][N]
    int64_t ldo;
    int out_f32, out_vec;    // out_vec: rows of out take 16-byte stores
    int add;                 // acc holds earlier pieces' sums
    int to_acc;              // store into acc rather than out
    float* acc;              // [M][N]
    const float* scale;      // null: 1
};

__device__ __constant__ int kPartA[6] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ int kPartB[6] = {0, 2, 1, 0, 1, 0};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Item { int m, n, split; };
__device__ __forceinline__ Item item_of(const GemmParams& p, int i) {
    Item it;
    const int tiles = p.n_m * p.n_n;
    it.split = i / tiles;
    i -= it.split * tiles;
    const int per = p.group * p.n_n, g = i / per;
    i -= g * per;
    const int gm = min(p.group, p.n_m - g * p.group);
    it.n = i / gm;
    it.m = g * p.group + (i - it.n * gm);
    return it;
}

// 32 consecutive values of a row as 16-bit pairs.
template <bool BF16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// A value as the sum of three bf16 parts.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    __nv_bfloat16 a = __float2bfloat16_rn(x);
    if (__hisinf(a) && !isinf(x)) a = __float2bfloat16_rz(x);
    p[0] = __bfloat162float(a);
    const float r = isfinite(p[0]) ? x - p[0] : 0.f;
    p[1] = __bfloat162float(__float2bfloat16_rn(r));
    p[2] = __bfloat162float(__float2bfloat16_rn(r - p[1]));
}

// ------------------------------------------------------------------ epilogues
// One 32-column chunk of an output row (this lane's) in v.
template <bool BF16>
__device__ __forceinline__ void store_out(const GemmParams& p, float (&v)[32], int row0, int row, int c0, int split,
                                          uint32_t* stage, int lane) {
    const bool live = row < p.M;
    const int n = p.N - c0;                                // valid columns from c0 on
    if (p.splits > 1 || p.to_acc) {
        // fp32 sums: of this split, or of the pieces so far.
        float* dst = p.splits > 1 ? static_cast<float*>(p.out) + ((int64_t)split * p.M + row) * p.N + c0
                                  : p.acc + (int64_t)row * p.N + c0;
        if (!live) return;
        if (n >= 32 && p.N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 t = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                if (p.splits == 1 && p.add) {
                    const float4 o = *reinterpret_cast<const float4*>(dst + i);
                    t.x += o.x; t.y += o.y; t.z += o.z; t.w += o.w;
                }
                *reinterpret_cast<float4*>(dst + i) = t;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n) dst[i] = v[i] + (p.splits == 1 && p.add ? dst[i] : 0.f);
        }
        return;
    }
    if (p.add && live) {
        const float* o = p.acc + (int64_t)row * p.N + c0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) v[i] += o[i];
    }
    const float s = p.scale ? *p.scale : 1.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= s;
    if (p.out_vec && n >= 32) {
        if (!live) return;
        if (p.out_f32) {
            float* dst = static_cast<float*>(p.out) + (int64_t)row * p.ldo + c0;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)row * p.ldo + c0;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(dst + i) =
                    make_uint4(pack2<BF16>(v[i], v[i + 1]), pack2<BF16>(v[i + 2], v[i + 3]),
                               pack2<BF16>(v[i + 4], v[i + 5]), pack2<BF16>(v[i + 6], v[i + 7]));
        }
        return;
    }
    // Rows off the 16-byte boundary, and the last columns: through shared
    // memory, so that a warp's stores run along a row.
    const int rows = min(32, p.M - row0);
    if (p.out_f32) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[lane * 17 + i] = __float_as_uint(v[half * 16 + i]);
            __syncwarp();
            const int c = half * 16 + (lane & 15);
            for (int r = lane >> 4; r < rows; r += 2)
                if (c < n)
                    static_cast<float*>(p.out)[(int64_t)(row0 + r) * p.ldo + c0 + c] =
                        __uint_as_float(stage[r * 17 + (lane & 15)]);
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) stage[lane * 17 + i] = pack2<BF16>(v[2 * i], v[2 * i + 1]);
        __syncwarp();
        for (int r = 0; r < rows; ++r)
            if (lane < n)
                static_cast<uint16_t*>(p.out)[(int64_t)(row0 + r) * p.ldo + c0 + lane] =
                    reinterpret_cast<const uint16_t*>(stage)[r * 34 + lane];
    }
}

template <bool BF16, int EPI, bool A_MN, bool B_MN, bool PROMOTE>
__global__ void __launch_bounds__(kThreads, 1)
ce_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int stage_bytes = kABytes + p.BN * kBK * 2;
    uint32_t* epi_stage = reinterpret_cast<uint32_t*>(smem + p.stages * stage_bytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes + kEpiWarps * kStageWarpBytes);
    // full[stages], empty[stages], accumulator full[2], empty[2], drain
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxRing + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto full_bar = [&](int i) { return smem_addr(&bars[i]); };
    auto empty_bar = [&](int i) { return smem_addr(&bars[kMaxRing + i]); };
    auto accf_bar = [&](int a) { return smem_addr(&bars[2 * kMaxRing + a]); };
    auto acce_bar = [&](int a) { return smem_addr(&bars[2 * kMaxRing + 2 + a]); };
    const uint32_t drain_bar = smem_addr(&bars[2 * kMaxRing + 4]);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < p.stages; ++i) { mbar_init(full_bar(i), 1); mbar_init(empty_bar(i), 1); }
        for (int a = 0; a < 2; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), kEpiWarps); }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&amap);
        tma_prefetch_desc(&bmap);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int items = p.n_m * p.n_n * p.splits, chunks = p.nk * p.pairs;
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
                const Item it = item_of(p, i);
                const int k0 = (int)((long long)chunks * it.split / p.splits);
                const int k1 = (int)((long long)chunks * (it.split + 1) / p.splits);
                const int m0 = it.m * kBM, n0 = it.n * p.BN;
                int pair = k0 / p.nk, k = k0 - pair * p.nk;
                for (int q = k0; q < k1; ++q) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1, abort_flag)) { ok = false; break; }
                    mbar_arrive_expect_tx(full_bar(stage), (uint32_t)stage_bytes);
                    const uint32_t a_dst = smem_addr(smem + stage * stage_bytes), b_dst = a_dst + kABytes;
                    const int ao = p.pairs > 1 ? kPartA[pair] * p.a_part : 0;
                    const int bo = p.pairs > 1 ? kPartB[pair] * p.b_part : 0;
                    if constexpr (A_MN) {
#pragma unroll
                        for (int j = 0; j < kBM / 64; ++j)
                            tma_load_2d(a_dst + j * 8192, &amap, full_bar(stage), ao + m0 + 64 * j, k * kBK);
                    } else {
                        tma_load_2d(a_dst, &amap, full_bar(stage), ao + k * kBK, m0);
                    }
                    if constexpr (B_MN) {
                        for (int j = 0; j < p.BN / 64; ++j)
                            tma_load_2d(b_dst + j * 8192, &bmap, full_bar(stage), bo + n0 + 64 * j, k * kBK);
                    } else {
                        tma_load_2d(b_dst, &bmap, full_bar(stage), bo + k * kBK, n0);
                    }
                    ++issued;
                    if (++stage == p.stages) { stage = 0; phase ^= 1; }
                    if (++k == p.nk) { k = 0; ++pair; }
                }
            }
            if (!ok) {
                // Let every copy already issued land before the CTA can exit.
                for (int i = 0; i < p.stages && i < issued; ++i) {
                    if (--stage < 0) { stage = p.stages - 1; phase ^= 1; }
                    mbar_drain_wait(full_bar(stage), phase);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc =
                umma_idesc_f16(BF16, kBM, p.BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued_any = false;
            for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
                const int split = i / (p.n_m * p.n_n);
                const int k0 = (int)((long long)chunks * split / p.splits);
                const int k1 = (int)((long long)chunks * (split + 1) / p.splits);
                for (int q0 = k0; q0 < k1 && ok;) {
                    const int q1 = PROMOTE ? min(k1, q0 + p.seg) : k1;
                    if (!mbar_wait(acce_bar(acc), acc_phase ^ 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * 256);
                    for (int q = q0; q < q1; ++q) {
                        if (!mbar_wait(full_bar(stage), phase, abort_flag)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a_addr = smem_addr(smem + stage * stage_bytes), b_addr = a_addr + kABytes;
                        // A K step of 16 elements: 32 bytes along a K-major row,
                        // 16 rows of 128 bytes of an MN-major block.
                        const uint64_t a_desc = A_MN ? sw128_mnmajor_desc(a_addr, 8192u) : sw128_kmajor_desc(a_addr);
                        const uint64_t b_desc = B_MN ? sw128_mnmajor_desc(b_addr, 8192u) : sw128_kmajor_desc(b_addr);
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            umma_f16(d_tmem, a_desc + (uint64_t)(k * (A_MN ? 128 : 2)),
                                     b_desc + (uint64_t)(k * (B_MN ? 128 : 2)), idesc, (q > q0 || k > 0) ? 1u : 0u);
                        issued_any = true;
                        umma_commit(empty_bar(stage));
                        if (++stage == p.stages) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    umma_commit(accf_bar(acc));
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                    q0 = q1;
                }
            }
            if (!ok && issued_any) {
                umma_commit(drain_bar);
                mbar_drain_wait(drain_bar, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Two groups of four warps share an accumulator's columns by halves;
        // warp q (mod 4) reads TMEM lanes 32 (q mod 4)..: one output row a lane.
        const int ew = warp - 2, half = ew >> 2, quarter = warp & 3;
        uint32_t* stage = epi_stage + ew * (kStageWarpBytes / 4);
        const int nch = p.BN / 32, c_lo = half ? (nch + 1) / 2 : 0, c_hi = half ? nch : (nch + 1) / 2;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const Item it = item_of(p, i);
            const int row0 = it.m * kBM + quarter * 32, row = row0 + lane, n0 = it.n * p.BN;
            const bool live = row < p.M;
            float m_run = -INFINITY, s_run = 0.f;              // EPI_LSE
            float lse = 0.f, coef = 0.f;                       // EPI_DZ
            int ty = -1;                                       // target's column in this piece
            if constexpr (EPI != EPI_OUT) {
                if (live) {
                    const int64_t t = p.target[row];
                    if (t != p.ignore && t >= 0 && t < p.vocab) ty = (int)t - p.col0;
                    if constexpr (EPI == EPI_DZ) {
                        lse = p.lse[row];
                        coef = p.coef[row];
                    }
                }
            }
            // PROMOTE: this warp's share of the tile's sums, in registers.
            constexpr int kKept = PROMOTE ? 4 : 1;             // 32-column chunks per warp at most
            float sum[kKept][32];
            if constexpr (PROMOTE) {
                const int k0 = (int)((long long)chunks * it.split / p.splits);
                const int k1 = (int)((long long)chunks * (it.split + 1) / p.splits);
#pragma unroll
                for (int c = 0; c < kKept; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
                bool got = true;
                for (int q0 = k0; q0 < k1; q0 += p.seg) {
                    got = __all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag));
                    if (!got) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll
                    for (int c = 0; c < kKept; ++c) {
                        if (c_lo + c < c_hi) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {      // 16 at a time: 128 sums leave few registers
                                uint32_t u[16];
                                tmem_ld_32x32b_x16(t_row + (c_lo + c) * 32 + e * 16, u);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) sum[c][e * 16 + j] += __uint_as_float(u[j]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acce_bar(acc));
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                }
                if (!got) break;
            } else {
                if (!__all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag))) break;
                tc_fence_after();
            }
            const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * 256);
            auto chunk = [&](int c, float (&v)[32]) {
                const int c0 = n0 + c * 32;                    // column within the piece
                const int n = p.N - c0;
                if constexpr (EPI == EPI_LSE) {
                    if (n < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= n) v[j] = -INFINITY;
                    }
                    float top = v[0];
#pragma unroll
                    for (int j = 1; j < 32; ++j) top = fmaxf(top, v[j]);
                    const float m_new = fmaxf(m_run, top);
                    // z - max first: a rounded max / ln 2 would scale the whole row.
                    const float base = m_new == -INFINITY ? 0.f : m_new;
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        s0 += exp2_approx((v[j] - base) * kLog2e);
                        s1 += exp2_approx((v[j + 1] - base) * kLog2e);
                    }
                    s_run = s_run * exp2_approx((m_run - base) * kLog2e) + (s0 + s1);
                    m_run = m_new;
                    if (ty >= c0 && ty < c0 + 32) {
                        const uint32_t hit = 1u << (ty - c0);  // a mask: an index would move v to memory
                        float z = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) z = hit & (1u << j) ? v[j] : z;
                        p.z_target[row] = z;
                    }
                } else if constexpr (EPI == EPI_DZ) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float d = exp2_approx((v[j] - lse) * kLog2e);
                        if (j == ty - c0) d -= 1.f;
                        // Ignored rows are zero whatever their logits are; so is the padding.
                        v[j] = coef != 0.f && j < n ? d * coef : 0.f;
                    }
                    if (live && c0 < p.dz_part) {              // the last tile may end past the piece
                        uint16_t* dst = static_cast<uint16_t*>(p.dz) + (int64_t)row * p.parts * p.dz_part + c0;
                        if (p.parts == 1) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                *reinterpret_cast<uint4*>(dst + j) =
                                    make_uint4(pack2<BF16>(v[j], v[j + 1]), pack2<BF16>(v[j + 2], v[j + 3]),
                                               pack2<BF16>(v[j + 4], v[j + 5]), pack2<BF16>(v[j + 6], v[j + 7]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float q[4][3];
#pragma unroll
                                for (int l = 0; l < 4; ++l) split3(v[j + l], q[l]);
#pragma unroll
                                for (int s = 0; s < 3; ++s)
                                    *reinterpret_cast<uint2*>(dst + (int64_t)s * p.dz_part + j) =
                                        make_uint2(pack2<true>(q[0][s], q[1][s]), pack2<true>(q[2][s], q[3][s]));
                            }
                        }
                    }
                } else {
                    if (n > 0) store_out<BF16>(p, v, row0, row, c0, it.split, stage, lane);
                }
            };
            if constexpr (PROMOTE) {
#pragma unroll
                for (int c = 0; c < kKept; ++c)
                    if (c_lo + c < c_hi) chunk(c_lo + c, sum[c]);
            } else {
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(t_row + c * 32, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[0][j] = __uint_as_float(u[j]);
                    chunk(c, sum[0]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce_bar(acc));
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
            if constexpr (EPI == EPI_LSE) {
                if (live && c_lo < c_hi)
                    p.lse_part[(int64_t)(2 * it.n + half) * p.M + row] = make_float2(m_run, s_run);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------ small kernels
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.f : top;
    s = s * exp2_approx((m - base) * kLog2e) + s2 * exp2_approx((m2 - base) * kLog2e);
    m = top;
}

// Sum over a block of 256 or 1024 threads, in every thread (fixed order).
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = lane_sum(v, 32);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int n = blockDim.x >> 5, lane = threadIdx.x & 31;
    return lane_sum(lane < n ? red[lane] : 0.f, 32);
}

__device__ __forceinline__ void reduce_losses(const float* row_loss, const int64_t* target, int n, int vocab,
                                              int64_t ignore, bool mean, float* loss, float* red) {
    float sum = 0.f, count = 0.f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t t = target[i];
        sum += row_loss[i];
        count += t != ignore && t >= 0 && t < vocab ? 1.f : 0.f;      // below 2^24 per thread: exact
    }
    sum = block_sum(sum, red);
    count = block_sum(count, red);
    if (threadIdx.x == 0) *loss = mean ? sum / fmaxf(count, 1.f) : sum;
}

// Join the tiles' (max, sum) pairs of `rows` rows per block (a power of two up
// to 32) by 256 / rows threads each.  A single block also reduces the losses.
__global__ void __launch_bounds__(256)
ce_rows_kernel(const float2* part, int tiles, int n, int rows, const float* z_target, const int64_t* target, int vocab,
               int64_t ignore, float* lse, float* row_loss, float* loss, int mean) {
    __shared__ float2 sh[256];
    __shared__ float red[32];
    pdl_wait();
    const int r = threadIdx.x % rows, k = threadIdx.x / rows, width = 256 / rows;
    const int row = blockIdx.x * rows + r;
    float m = -INFINITY, s = 0.f;
    if (row < n) {
#pragma unroll 4
        for (int i = k; i < tiles; i += width) {
            const float2 v = part[(int64_t)i * n + row];
            join(m, s, v.x, v.y);
        }
    }
    sh[threadIdx.x] = make_float2(m, s);
    for (int w = width >> 1; w > 0; w >>= 1) {
        __syncthreads();
        if (k < w) {
            const float2 v = sh[threadIdx.x + w * rows];
            join(m, s, v.x, v.y);
            sh[threadIdx.x] = make_float2(m, s);
        }
    }
    if (k == 0 && row < n) {
        const float l = m + logf(s);
        lse[row] = l;
        const int64_t t = target[row];
        row_loss[row] = t == ignore ? 0.f : (t < 0 || t >= vocab ? nanf("") : l - z_target[row]);
    }
    if (loss && gridDim.x == 1) {
        __syncthreads();
        reduce_losses(row_loss, target, n, vocab, ignore, mean, loss, red);
    }
}

__global__ void __launch_bounds__(1024) ce_reduce_kernel(const float* row_loss, const int64_t* target, int n, int vocab,
                                                         int64_t ignore, int mean, float* loss) {
    __shared__ float red[32];
    pdl_wait();
    reduce_losses(row_loss, target, n, vocab, ignore, mean, loss, red);
}

// g_n = coef[n] * common.  Sum and mean: coef is 2^14 for the rows that count
// (|dz| <= 1) and common holds dloss (over their number for the mean).  None:
// coef is dloss scaled by a power of two, the largest in [2^14, 2^15).  Rows
// that do not count have coef 0.
__global__ void __launch_bounds__(1024) ce_coef_kernel(const float* dloss, const int64_t* target, int n, int vocab,
                                                       int64_t ignore, int per_row, int mean, float* coef,
                                                       float* common) {
    __shared__ float red[32];
    __shared__ float up_s;
    pdl_wait();
    float count = 0.f, top = 0.f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t t = target[i];
        if (t != ignore && t >= 0 && t < vocab) {
            count += 1.f;
            if (per_row) top = fmaxf(top, fabsf(dloss[i]));
        }
    }
    count = block_sum(count, red);
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) top = fmaxf(top, red[i]);
        int e = 14;
        if (per_row) {
            e = 0;
            if (top > 0.f && isfinite(top)) {
                frexpf(top, &e);                   // top = f 2^e, f in [0.5, 1)
                e = 15 - e;
                e = e > 126 ? 126 : (e < -126 ? -126 : e);
            }
        }
        up_s = ldexpf(1.f, e);
        const float g = per_row ? 1.f : (mean ? *dloss / fmaxf(count, 1.f) : *dloss);
        *common = g * ldexpf(1.f, -e);
    }
    __syncthreads();
    const float up = up_s;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t t = target[i];
        const bool in = t != ignore && t >= 0 && t < vocab;
        coef[i] = in ? (per_row ? dloss[i] * up : up) : 0.f;
    }
}

// Rows of T as [rows][parts * pitch] 16-bit values for the tensor cores, zero
// past `cols`, and zero for rows whose target does not count (skip given):
// their weight in dw is zero, which would not hide a NaN.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256) ce_pack_kernel(const T* src, int64_t stride, int64_t rows, int cols, int pitch,
                                                      int vec, const int64_t* target, int vocab, int64_t ignore,
                                                      uint16_t* dst) {
    pdl_wait();
    const int per = pitch / 8;
    const int64_t total = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        bool keep = true;
        if (target) {
            const int64_t t = target[row];
            keep = t != ignore && t >= 0 && t < vocab;
        }
        const T* s = src + row * stride + c;
        uint16_t* d = dst + row * (int64_t)PARTS * pitch + c;
        if constexpr (PARTS == 1) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (keep) {
                if (vec && c + 8 <= cols) {
                    v = *reinterpret_cast<const uint4*>(s);
                } else {
                    uint16_t e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = c + j < cols ? reinterpret_cast<const uint16_t*>(s)[j] : 0;
                    v = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                   e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                }
            }
            *reinterpret_cast<uint4*>(d) = v;
        } else {
            float q[8][3];
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(keep && c + j < cols ? to_f32(s[j]) : 0.f, q[j]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4*>(d + (int64_t)k * pitch) =
                    make_uint4(pack2<true>(q[0][k], q[1][k]), pack2<true>(q[2][k], q[3][k]),
                               pack2<true>(q[4][k], q[5][k]), pack2<true>(q[6][k], q[7][k]));
        }
    }
}

// out = scale (acc + sum over splits), or acc = that sum unscaled (to_acc).
template <typename T>
__global__ void __launch_bounds__(256) ce_join_kernel(const float* part, int splits, int64_t count, float* acc, int add,
                                                      int to_acc, const float* scale, T* out) {
    pdl_wait();
    const float s = *scale;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += (int64_t)gridDim.x * blockDim.x) {
        float v = add ? acc[i] : 0.f;
#pragma unroll 4
        for (int k = 0; k < splits; ++k) v += part[(int64_t)k * count + i];
        if (to_acc) acc[i] = v;
        else out[i] = from_f32<T>(v * s);
    }
}

// ------------------------------------------------------------------ host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef CUresult (*PFN_encode_t)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A row-major 16-bit matrix read in boxes of 64 columns (128 bytes, swizzled)
// by `box_rows` rows; zeros outside.
bool make_map(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    static PFN_encode_t enc = reinterpret_cast<PFN_encode_t>(driver_entry("cuTensorMapEncodeTiled"));
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t str[1] = {(cuuint64_t)pitch * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
               const_cast<void*>(base), dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kMostPiece = 1LL << 28;      // three parts of a piece keep 32-bit column numbers


// Tile width and K splits by an estimate in SM cycles.  An item (one tile of
// one split) takes its MMAs (2 BN cycles per 64-wide chunk), a fixed cost per
// chunk (barriers; more of it shows with narrow tiles) and a fixed cost per
// item (pipeline fill, the last epilogue); items run in waves over the SMs;
// splits add the write and read of their fp32 sums and one launch.
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t chunks, int step, bool may_split) {
    const int sms = device_sm_count();
    GemmPlan best{256, 1};
    double best_t = -1;
    for (int bn = 256; bn >= 64; bn -= step) {
        if (bn > 64 && bn - step >= N) continue;             // wider than the output needs
        const int64_t tiles = ceil_div(M, kBM) * ceil_div(N, bn);
        for (int s = 1; s <= 64 && s <= chunks; s = s < 4 ? s + 1 : s + s / 2) {
            if (s > 1 && !may_split) break;
            const double waves = (double)ceil_div(tiles * s, sms);
            double t = waves * ((double)ceil_div(chunks, s) * (2.0 * bn + 64.0) + 3000.0);
            if (s > 1) t += 4000.0 + (double)s * M * N * 8.0 / 3500.0;
            if (best_t < 0 || t < best_t * 0.999) { best_t = t; best = GemmPlan{bn, s}; }
        }
    }
    return best;
}

// Chunks per accumulation: 256 K elements, 16 steps.  The epilogue's additions
// (32 columns in about 100 cycles a warp) stay under those chunks' MMAs.
constexpr int kSegment = 4;

// Lift a kernel's shared-memory limit, once per device and kernel.
bool allow_smem(const void* kern) {
    static std::mutex lock;
    static std::set<std::pair<int, const void*>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> hold(lock);
    if (done.count({dev, kern})) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess) return false;
    done.insert({dev, kern});
    return true;
}

template <int EPI, bool A_MN, bool B_MN>
conv2d_status launch_gemm(bool bf16, const CUtensorMap& a, const CUtensorMap& b, GemmParams p, cudaStream_t st) {
    // fp32 operands (six products) are bf16 parts; their results stay in fp32.
    auto kern = p.pairs > 1 ? ce_gemm_kernel<true, EPI, A_MN, B_MN, true>
                : bf16      ? ce_gemm_kernel<true, EPI, A_MN, B_MN, EPI == EPI_LSE>
                            : ce_gemm_kernel<false, EPI, A_MN, B_MN, EPI == EPI_LSE>;
    p.seg = kSegment;
    const int stage_bytes = kABytes + p.BN * kBK * 2;
    const int fixed = 1024 + kEpiWarps * kStageWarpBytes + (2 * kMaxRing + 5) * 8 + 16;
    p.stages = (kSmemMost - fixed) / stage_bytes;
    if (p.stages > kMaxRing) p.stages = kMaxRing;
    const int smem = fixed + p.stages * stage_bytes;
    if (!allow_smem(reinterpret_cast<const void*>(kern))) return CONV2D_ERR_CUDA;
    p.n_m = (int)ceil_div(p.M, kBM);
    p.n_n = (int)ceil_div(p.N, p.BN);
    const int64_t items = (int64_t)p.n_m * p.n_n * p.splits;
    const int sms = device_sm_count();
    const int grid = items < sms ? (int)items : sms;
    // Row tiles whose A (read again for every column tile) stays in the L2 beside the streams.
    const int64_t a_tile = (int64_t)kBM * p.nk * kBK * 2 * (p.pairs > 1 ? 3 : 1);
    int64_t g = (24 << 20) / a_tile;
    p.group = (int)(g < 1 ? 1 : (g > p.n_m ? p.n_m : g));
    return launch_after(kern, dim3(grid), dim3(kThreads), smem, st, a, b, p) == cudaSuccess ? CONV2D_OK
                                                                                            : CONV2D_ERR_CUDA;
}

void take(size_t& at, size_t& off, size_t bytes) {
    off = at;
    at += align_up(bytes, 1024);
}

CePlan plan_ce(const linear_ce_desc& d, bool backward) {
    CePlan c{};
    const bool f32 = d.dtype == CONV2D_F32;
    c.bf16 = d.dtype != CONV2D_F16;
    c.parts = f32 ? 3 : 1;
    c.pairs = f32 ? 6 : 1;
    c.pack_w = f32 || d.ws % 8 != 0;
    // The backward pass always copies h: ignored rows must be zero in dw's product.
    c.pack_h = backward || f32 || d.hs % 8 != 0;
    c.dp = ceil_div(d.hidden, 64) * 64;
    // Pieces: the forward pass needs them only for the packed copy of w.
    const int64_t budget = 256LL << 20;
    int64_t piece = ceil_div(d.vocab, 256) * 256;
    if (backward || c.pack_w) {
        int64_t most = budget;
        if (backward) most = budget / (d.tokens * 2 * c.parts);
        if (c.pack_w && budget / (c.dp * 2 * c.parts) < most) most = budget / (c.dp * 2 * c.parts);
        if (d.piece > 0 && backward) most = (d.piece < kMostPiece ? d.piece : kMostPiece) + 255;
        most = most / 256 * 256;
        if (most < 256) most = 256;
        if (piece > most) piece = most;
        piece = ceil_div(ceil_div(d.vocab, ceil_div(d.vocab, piece)), 256) * 256;      // even pieces
    }
    c.piece = piece;
    c.pieces = ceil_div(d.vocab, piece);
    const int64_t nk = c.dp / 64;
    const int64_t v = d.vocab < piece ? d.vocab : piece;
    // dz is read in 64-column chunks, so its tiles write whole ones (zeros past the vocabulary).
    c.z = plan_gemm(d.tokens, v, nk * c.pairs, backward ? 64 : 32, false);
    size_t at = 0;
    if (!backward) {
        take(at, c.part, (size_t)d.tokens * 2 * (size_t)(c.pieces * ceil_div(v, c.z.BN)) * sizeof(float2));
        take(at, c.z_target, (size_t)d.tokens * 4);
        take(at, c.row_loss, (size_t)d.tokens * 4);
    } else {
        c.dh = plan_gemm(d.tokens, d.hidden, ceil_div(v, 64) * c.pairs, 64, true);
        c.dw = plan_gemm(v, d.hidden, ceil_div(d.tokens, 64) * c.pairs, 64, true);
        take(at, c.coef, (size_t)d.tokens * 4);
        take(at, c.common, 4);
        take(at, c.dz, (size_t)d.tokens * (size_t)piece * 2 * c.parts);
        if (c.pieces > 1) take(at, c.acc, (size_t)d.tokens * d.hidden * 4);
        size_t sums = 0;
        if (c.dh.splits > 1) sums = (size_t)c.dh.splits * d.tokens * d.hidden * 4;
        if (c.dw.splits > 1 && (size_t)c.dw.splits * v * d.hidden * 4 > sums)
            sums = (size_t)c.dw.splits * v * d.hidden * 4;
        take(at, c.sums, sums);
    }
    if (c.pack_h) take(at, c.hp, (size_t)d.tokens * c.dp * 2 * c.parts);
    if (c.pack_w) take(at, c.wp, (size_t)v * c.dp * 2 * c.parts);
    c.total = at;
    return c;
}

cudaError_t pack(const linear_ce_desc& d, const void* src, int64_t stride, int64_t rows, int64_t dp, const int64_t* target,
                 void* dst, cudaStream_t st) {
    const int64_t work = ceil_div(rows * (dp / 8), 256);
    const int64_t most = (int64_t)device_sm_count() * 16;
    const dim3 grid((unsigned)(work < most ? work : most)), block(256);
    if (d.dtype == CONV2D_F32)
        return launch_after(ce_pack_kernel<float, 3>, grid, block, 0, st, static_cast<const float*>(src), stride, rows,
                            (int)d.hidden, (int)dp, 0, target, (int)d.vocab, d.ignore_index,
                            static_cast<uint16_t*>(dst));
    const int vec = stride % 8 == 0 && aligned_to(src, 16);
    return launch_after(ce_pack_kernel<__half, 1>, grid, block, 0, st, static_cast<const __half*>(src), stride, rows,
                        (int)d.hidden, (int)dp, vec, target, (int)d.vocab, d.ignore_index, static_cast<uint16_t*>(dst));
}

// h and w as the tensor cores read them: base, columns and row pitch.
struct Operand { const void* base; int64_t cols, pitch; };

conv2d_status gemm_z(const CePlan& c, const linear_ce_desc& d, int epi, const Operand& h, const Operand& w, int64_t rows_w,
                     GemmParams p, cudaStream_t st) {
    p.M = (int)d.tokens;
    p.N = (int)rows_w;
    p.BN = c.z.BN;
    p.nk = (int)(c.dp / 64);
    p.pairs = c.pairs;
    p.a_part = p.b_part = (int)c.dp;
    p.splits = 1;
    p.vocab = (int)d.vocab;
    p.ignore = d.ignore_index;
    CUtensorMap a, b;
    if (!make_map(&a, h.base, c.bf16, d.tokens, h.cols, h.pitch, kBM) ||
        !make_map(&b, w.base, c.bf16, rows_w, w.cols, w.pitch, p.BN))
        return CONV2D_ERR_CUDA;
    return epi == EPI_LSE ? launch_gemm<EPI_LSE, false, false>(c.bf16, a, b, p, st)
                          : launch_gemm<EPI_DZ, false, false>(c.bf16, a, b, p, st);
}

template <typename T>
cudaError_t join_splits(const float* part, int splits, int64_t count, float* acc, int add, int to_acc,
                        const float* scale, void* out, cudaStream_t st) {
    const int64_t work = ceil_div(count, 256), most = (int64_t)device_sm_count() * 16;
    return launch_after(ce_join_kernel<T>, dim3((unsigned)(work < most ? work : most)), dim3(256), 0, st, part, splits,
                        count, acc, add, to_acc, scale, static_cast<T*>(out));
}

// out = scale (acc + A B^T), split over K when planned; A is K-major (dz for
// dh) or MN-major (dz for dw), B is MN-major.
template <bool A_MN>
conv2d_status gemm_out(const CePlan& c, const linear_ce_desc& d, const GemmPlan& g, const CUtensorMap& a,
                       const CUtensorMap& b, int64_t M, int64_t K, int a_part, int b_part, void* out, float* acc,
                       int add, int to_acc, const float* scale, float* sums, cudaStream_t st) {
    GemmParams p{};
    p.M = (int)M;
    p.N = (int)d.hidden;
    p.BN = g.BN;
    p.nk = (int)ceil_div(K, 64);
    p.pairs = c.pairs;
    p.a_part = a_part;
    p.b_part = b_part;
    p.splits = g.splits < p.nk * p.pairs ? g.splits : p.nk * p.pairs;
    p.ldo = d.hidden;
    p.out_f32 = d.dtype == CONV2D_F32;
    p.out_vec = d.hidden * (p.out_f32 ? 4 : 2) % 16 == 0 && aligned_to(out, 16);
    p.add = add;
    p.to_acc = to_acc;
    p.acc = acc;
    p.scale = scale;
    p.out = p.splits > 1 ? sums : out;
    const conv2d_status s = launch_gemm<EPI_OUT, A_MN, true>(c.bf16, a, b, p, st);
    if (s != CONV2D_OK || p.splits == 1) return s;
    cudaError_t e;
    switch (d.dtype) {
        case CONV2D_F32: e = join_splits<float>(sums, p.splits, M * d.hidden, acc, add, to_acc, scale, out, st); break;
        case CONV2D_F16: e = join_splits<__half>(sums, p.splits, M * d.hidden, acc, add, to_acc, scale, out, st); break;
        default:
            e = join_splits<__nv_bfloat16>(sums, p.splits, M * d.hidden, acc, add, to_acc, scale, out, st);
    }
    return e == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

const void* at_row(const void* base, int64_t row, int64_t stride, size_t e) {
    return static_cast<const uint8_t*>(base) + (size_t)(row * stride) * e;
}

}  // namespace

void linear_ce_plan(linear_ce_desc& d) {
    d.fwd = d.bwd = CePlan{};
    if (d.tokens == 0) return;
    d.fwd = plan_ce(d, false);
    d.bwd = plan_ce(d, true);
}

conv2d_status launch_linear_ce_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                                   float* loss, float* lse, void* ws, cudaStream_t st) {
    const CePlan& c = d.fwd;
    uint8_t* base = static_cast<uint8_t*>(ws);
    const size_t e = elem_bytes(d.dtype);
    Operand ho{h, d.hidden, d.hs};
    if (c.pack_h) {
        if (pack(d, h, d.hs, d.tokens, c.dp, nullptr, base + c.hp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
        ho = Operand{base + c.hp, c.dp * c.parts, c.dp * c.parts};
    }
    GemmParams p{};
    p.target = target;
    p.z_target = reinterpret_cast<float*>(base + c.z_target);
    float2* part = reinterpret_cast<float2*>(base + c.part);
    int tiles = 0;
    for (int64_t v0 = 0; v0 < d.vocab; v0 += c.piece) {
        const int64_t rows = d.vocab - v0 < c.piece ? d.vocab - v0 : c.piece;
        Operand wo{at_row(w, v0, d.ws, e), d.hidden, d.ws};
        if (c.pack_w) {
            if (pack(d, wo.base, d.ws, rows, c.dp, nullptr, base + c.wp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
            wo = Operand{base + c.wp, c.dp * c.parts, c.dp * c.parts};
        }
        p.col0 = (int)v0;
        p.lse_part = part + (size_t)tiles * d.tokens;
        const conv2d_status s = gemm_z(c, d, EPI_LSE, ho, wo, rows, p, st);
        if (s != CONV2D_OK) return s;
        tiles += 2 * (int)ceil_div(rows, c.z.BN);
    }
    float* row_loss = d.reduction == HEAD_REDUCE_NONE ? loss : reinterpret_cast<float*>(base + c.row_loss);
    float* total = d.reduction == HEAD_REDUCE_NONE ? nullptr : loss;
    int rows = 1;
    while (rows < 32 && rows < d.tokens) rows *= 2;
    const unsigned grid = (unsigned)ceil_div(d.tokens, rows);
    const int mean = d.reduction == HEAD_REDUCE_MEAN;
    if (launch_after(ce_rows_kernel, dim3(grid), dim3(256), 0, st, static_cast<const float2*>(part), tiles,
                     (int)d.tokens, rows, static_cast<const float*>(p.z_target), target, (int)d.vocab, d.ignore_index,
                     lse, row_loss, total, mean) != cudaSuccess)
        return CONV2D_ERR_CUDA;
    if (total && grid > 1 &&
        launch_after(ce_reduce_kernel, dim3(1), dim3(1024), 0, st, static_cast<const float*>(row_loss), target,
                     (int)d.tokens, (int)d.vocab, d.ignore_index, mean, total) != cudaSuccess)
        return CONV2D_ERR_CUDA;
    return CONV2D_OK;
}

conv2d_status launch_linear_ce_bwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                                   const float* lse, const float* dloss, void* dh, void* dw, void* ws,
                                   cudaStream_t st) {
    const CePlan& c = d.bwd;
    uint8_t* base = static_cast<uint8_t*>(ws);
    const size_t e = elem_bytes(d.dtype);
    float* coef = reinterpret_cast<float*>(base + c.coef);
    float* common = reinterpret_cast<float*>(base + c.common);
    float* acc = c.pieces > 1 ? reinterpret_cast<float*>(base + c.acc) : nullptr;
    float* sums = reinterpret_cast<float*>(base + c.sums);
    if (launch_after(ce_coef_kernel, dim3(1), dim3(1024), 0, st, dloss, target, (int)d.tokens, (int)d.vocab,
                     d.ignore_index, d.reduction == HEAD_REDUCE_NONE ? 1 : 0, d.reduction == HEAD_REDUCE_MEAN ? 1 : 0,
                     coef, common) != cudaSuccess)
        return CONV2D_ERR_CUDA;
    if (pack(d, h, d.hs, d.tokens, c.dp, target, base + c.hp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
    const Operand ho{base + c.hp, c.dp * c.parts, c.dp * c.parts};
    GemmParams p{};
    p.target = target;
    p.lse = lse;
    p.coef = coef;
    p.dz = base + c.dz;
    p.dz_part = (int)c.piece;
    p.parts = c.parts;
    for (int64_t v0 = 0; v0 < d.vocab; v0 += c.piece) {
        const int64_t rows = d.vocab - v0 < c.piece ? d.vocab - v0 : c.piece;
        const bool first = v0 == 0, last = v0 + rows >= d.vocab;
        Operand wo{at_row(w, v0, d.ws, e), d.hidden, d.ws};
        if (c.pack_w) {
            if (pack(d, wo.base, d.ws, rows, c.dp, nullptr, base + c.wp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
            wo = Operand{base + c.wp, c.dp * c.parts, c.dp * c.parts};
        }
        p.col0 = (int)v0;
        conv2d_status s = gemm_z(c, d, EPI_DZ, ho, wo, rows, p, st);
        if (s != CONV2D_OK) return s;
        CUtensorMap a, b;
        const int64_t dz_pitch = c.piece * c.parts;
        if (dh) {
            if (!make_map(&a, p.dz, c.bf16, d.tokens, dz_pitch, dz_pitch, kBM) ||
                !make_map(&b, wo.base, c.bf16, rows, wo.cols, wo.pitch, 64))
                return CONV2D_ERR_CUDA;
            s = gemm_out<false>(c, d, c.dh, a, b, d.tokens, rows, (int)c.piece, (int)c.dp, dh, acc, !first, !last, common,
                                sums, st);
            if (s != CONV2D_OK) return s;
        }
        if (dw) {
            if (!make_map(&a, p.dz, c.bf16, d.tokens, dz_pitch, dz_pitch, 64) ||
                !make_map(&b, ho.base, c.bf16, d.tokens, ho.cols, ho.pitch, 64))
                return CONV2D_ERR_CUDA;
            s = gemm_out<true>(c, d, c.dw, a, b, rows, d.tokens, (int)c.piece, (int)c.dp,
                               static_cast<uint8_t*>(dw) + (size_t)v0 * d.hidden * e, nullptr, 0, 0, common, sums, st);
            if (s != CONV2D_OK) return s;
        }
    }
    return CONV2D_OK;
}

cudaError_t status_read_clear_ce(cudaStream_t st, uint32_t* out) { return status_read_clear(st, out); }
cudaError_t wait_limit_set_ce(cudaStream_t st, uint64_t ns) { return wait_limit_set(st, ns); }

}  // namespace conv2d_gb300
