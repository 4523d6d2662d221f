// Linear cross entropy over a large vocabulary, forward and backward, on the
// 5th-generation tensor cores (tcgen05 MMA, accumulators in tensor memory,
// operands fed by TMA).
//
//   forward    z = h w^T one 128 x BN tile at a time; the epilogue reduces
//              each row of the tile to (max, sum exp(z - max)) and picks the
//              target's z, so z never reaches memory.  A second kernel joins
//              the tiles' pairs: the maximum first, then the rescaled sums.
//   backward   per piece of the vocabulary: z again, turned by the epilogue
//              into dz = g (exp(z - lse) - [v = y]) in 16 bits (twice 16 for up
//              to 256 rows); then dh += dz w and dw = dz^T h.
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
// grows with K.  Where the result is kept in fp32 (the losses, and everything of
// fp32 operands), and for dz of long 16-bit rows (promote_z), the accumulator
// therefore runs for `seg` chunks only and the epilogue adds these partial sums
// in registers, rounded to nearest, while the next ones are computed (PROMOTE).
//
// Large products run on CTA pairs (PAIR): the tile is 256 rows by BN columns,
// each CTA keeps half of the rows of A and half of the columns of B in its
// shared memory and the accumulators of its rows, and one MMA reads both, so a
// CTA's copies and shared-memory reads per product are a third less.
//
// Few rows by many columns (or a long K by a small output) is split over K and
// joined by a second kernel in a fixed order, so that all SMs have work.  Few
// tokens go to linear_ce_few.cu instead.
//
// Measured (products counted once): the logits with their reduction 1.51 PFLOP/s
// at 4096 x 1024 x 65536 bf16 and 1.76 at 16384 x 2048 x 65536, dz 1.40 and 1.55,
// dh and dw 1.4 to 1.6; large calls run at the power limit (clock 1.5 GHz of
// 2.07).  fp32 1000 x 768 x 20011: losses 140 us, dz 200 us, dh and dw 300 us (1.3,
// 0.9 and 1.2 PFLOP/s of the six products): dz's three parts leave at each
// tile's end, longer than two accumulators cover.
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "head_device.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

constexpr int kBM = 128, kBK = 64;            // MMA rows; K elements per stage (128 bytes)
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxRing = 8;
// Epilogue warps.  PROMOTE: sixteen, so that a segment's sums are out of tensor
// memory well within the next segment's MMAs (eight took 2400 cycles for 2048).
__host__ __device__ constexpr int epi_warps(bool promote) { return promote ? 16 : 8; }
constexpr int kStageWarpBytes = 32 * 17 * 4;  // epilogue staging per warp: 32 rows of 17 words
constexpr int kSmemMost = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f;

enum Epilogue { EPI_LSE = 0, EPI_DZ = 1, EPI_OUT = 2 };

struct GemmParams {
    int M, N;                // valid extents of C
    int a_mn;                // A is MN-major
    int n_m, n_n;            // tiles
    int group;               // row tiles that share each column tile before the next one is taken
    int nk, pairs;           // K chunks of one product of parts, and such products (1, 2 or 6)
    int a_part, b_part;      // column offset from one part to the next
    int splits;
    // EPI_LSE and EPI_DZ
    int col0;                // first vocabulary row of this piece
    int vocab;
    int64_t ignore;
    const int64_t* target;
    float2* lse_part;        // [column tile][M]
    float* z_target;         // [M]
    const float *lse, *coef; // [M]
    void* dz;                // [M][parts * dz_part]
    int dz_part, parts;
    // EPI_OUT
    void* out;               // final element type, or the fp32 partial sums [split][M][lds]
    int64_t ldo;
    int out_f32, out_vec;    // out_vec: rows of out take 32-byte (2), 16-byte (1) or no wide stores (0)
    int64_t lds;             // row pitch of the fp32 sums: a multiple of 64, so they always move whole
    int add;                 // acc holds earlier pieces' sums
    int to_acc;              // store into acc rather than out
    float* acc;              // [M][lds]
    const float* scale;      // null: 1
};

// A launch: one product, or two that share the machine (dh and dw: the items of
// the first, longer ones come first, those of the second fill its last wave).
struct GemmJobs {
    GemmParams job[2];
    int items0, items;       // items of the first product, and of both
    int BN;                  // tile width
    int stages, seg;         // ring depth; PROMOTE: chunks per accumulation in tensor memory
    int epi_bytes;           // epilogue staging in shared memory (0: none needed)
};
struct GemmMaps { CUtensorMap a[2], b[2]; };

__device__ __constant__ int kPartA[6] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ int kPartB[6] = {0, 2, 1, 0, 1, 0};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Join two (max, sum of exp(z - max)) pairs.  A maximum that is infinite is not taken
// out: its sum is 0 or infinite as it stands, where inf - inf would make it NaN.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float base = isinf(top) ? 0.f : top;
    s = s * exp2_approx((m - base) * kLog2e) + s2 * exp2_approx((m2 - base) * kLog2e);
    m = top;
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

template <bool BF16> __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    unpack2f(widen_pair<std::conditional_t<BF16, __nv_bfloat16, __half>>(w), a, b);
}

// The bf16 nearest to x (toward zero where that would overflow), and what is
// left for the next part: three parts hold all 24 bits of a float.
__device__ __forceinline__ float part_of(float x) {
    __nv_bfloat16 a = __float2bfloat16_rn(x);
    if (__hisinf(a) && !isinf(x)) a = __float2bfloat16_rz(x);
    return __bfloat162float(a);
}
__device__ __forceinline__ float rest_of(float x, float part) { return isfinite(part) ? x - part : 0.f; }
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    p[0] = part_of(x);
    x = rest_of(x, p[0]);
    p[1] = part_of(x);
    p[2] = part_of(rest_of(x, p[1]));
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
        float* dst = p.splits > 1 ? static_cast<float*>(p.out) + ((int64_t)split * p.M + row) * p.lds + c0
                                  : p.acc + (int64_t)row * p.lds + c0;
        if (!live || c0 >= p.lds) return;
        if (p.splits == 1 && p.add) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 o = *reinterpret_cast<const float4*>(dst + i);
                v[i] += o.x; v[i + 1] += o.y; v[i + 2] += o.z; v[i + 3] += o.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
            st_global_v8(dst + i, w);
        }
        return;
    }
    if (p.add && live) {                                   // (the sums' rows are whole chunks)
        const float* o = p.acc + (int64_t)row * p.lds + c0;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 t = *reinterpret_cast<const float4*>(o + i);
            v[i] += t.x; v[i + 1] += t.y; v[i + 2] += t.z; v[i + 3] += t.w;
        }
    }
    const float s = p.scale ? *p.scale : 1.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= s;
    if (p.out_vec && n >= 32) {
        if (!live) return;
        if (p.out_f32) {
            float* dst = static_cast<float*>(p.out) + (int64_t)row * p.ldo + c0;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
                if (p.out_vec == 2) {
                    st_global_v8(dst + i, w);
                } else {
                    *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(dst + i + 4) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        } else {
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)row * p.ldo + c0;
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack2<BF16>(v[i + 2 * j], v[i + 2 * j + 1]);
                if (p.out_vec == 2) {
                    st_global_v8(dst + i, w);
                } else {
                    *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(dst + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
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

template <bool BF16, int EPI, bool PROMOTE, bool PAIR>
__global__ void __launch_bounds__(32 * (2 + epi_warps(PROMOTE)), 1)
ce_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmJobs jobs) {
    constexpr bool B_MN = EPI == EPI_OUT;
    constexpr int kEpiWarps = epi_warps(PROMOTE), kGroups = kEpiWarps / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    constexpr int kTileM = PAIR ? 2 * kBM : kBM, kCtas = PAIR ? 2 : 1;
    const int rank = PAIR ? (int)cluster_rank() : 0;       // 0 issues the pair's MMAs
    const int bn = PAIR ? jobs.BN / 2 : jobs.BN;           // columns of B in this CTA
    const int stages = jobs.stages, stage_bytes = kABytes + bn * kBK * 2;
    uint32_t* epi_stage = reinterpret_cast<uint32_t*>(smem + stages * stage_bytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes + jobs.epi_bytes);
    // full[stages], empty[stages], accumulator full[2], empty[2], drain
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxRing + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* copies = abort_flag + 1;                 // PAIR: ring fills that this CTA has issued
    volatile int* peer = copies + 1;                       // PAIR: the other CTA's two words, which it writes here
    auto full_bar = [&](int i) { return smem_addr(&bars[i]); };
    auto empty_bar = [&](int i) { return smem_addr(&bars[kMaxRing + i]); };
    auto accf_bar = [&](int a) { return smem_addr(&bars[2 * kMaxRing + a]); };
    auto acce_bar = [&](int a) { return smem_addr(&bars[2 * kMaxRing + 2 + a]); };
    const uint32_t drain_bar = smem_addr(&bars[2 * kMaxRing + 4]);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < stages; ++i) { mbar_init(full_bar(i), 1); mbar_init(empty_bar(i), 1); }
        for (int a = 0; a < 2; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), kCtas * kEpiWarps); }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *copies = 0;
        mbar_fence_init();
        tma_prefetch_desc(&maps.a[0]);
        tma_prefetch_desc(&maps.b[0]);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), 512);
        } else {
            tmem_alloc(smem_addr(tmem_slot), 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();                    // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    // Items are dealt out in turn; every role walks them alike.
    const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;
    auto job_of = [&](int& i) {                            // product of item i, which becomes its number there
        if (EPI != EPI_OUT || i < jobs.items0) return 0;
        i -= jobs.items0;
        return 1;
    };
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            for (int n_item = first; n_item < jobs.items && ok; n_item += step) {
                int i = n_item;
                const int j = job_of(i);
                const GemmParams& p = jobs.job[j];
                const CUtensorMap *amap = &maps.a[j], *bmap = &maps.b[j];
                const Item it = item_of(p, i);
                const int chunks = p.nk * p.pairs;
                const int k0 = (int)((long long)chunks * it.split / p.splits);
                const int k1 = (int)((long long)chunks * (it.split + 1) / p.splits);
                const int m0 = it.m * kTileM + rank * kBM, n0 = it.n * jobs.BN + rank * bn;
                const int nk = p.nk, a_mn = p.a_mn, pairs = p.pairs;
                // Six products run one after the other; two (never PROMOTE) in turn,
                // the second part first, B's chunk read again from the L2.
                const int other = !PROMOTE && pairs == 2 ? p.a_part : 0;
                int pair = k0 / nk, k = k0 - pair * nk, ao = 0, bo = 0;
                if (!PROMOTE && pairs == 2) {
                    k = k0 >> 1;
                    ao = k0 & 1 ? 0 : other;
                }
                for (int q = k0; q < k1; ++q) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1, abort_flag)) { ok = false; break; }
                    // A pair's copies all count on the issuing CTA's barrier.
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), (uint32_t)(kCtas * stage_bytes));
                    const uint32_t bar = PAIR ? cluster_addr(full_bar(stage), 0) : full_bar(stage);
                    const uint32_t a_dst = smem_addr(smem + stage * stage_bytes), b_dst = a_dst + kABytes;
                    if (PROMOTE) {
                        ao = pairs > 1 ? kPartA[pair] * p.a_part : 0;
                        bo = pairs > 1 ? kPartB[pair] * p.b_part : 0;
                    }
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
                        if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, c0, c1);
                        else                tma_load_2d(dst, map, bar, c0, c1);
                    };
                    if (EPI == EPI_OUT && a_mn) {
#pragma unroll
                        for (int l = 0; l < kBM / 64; ++l) load(a_dst + l * 8192, amap, ao + m0 + 64 * l, k * kBK);
                    } else {
                        load(a_dst, amap, ao + k * kBK, m0);
                    }
                    if constexpr (B_MN) {
                        for (int l = 0; l < bn / 64; ++l) load(b_dst + l * 8192, bmap, bo + n0 + 64 * l, k * kBK);
                    } else {
                        load(b_dst, bmap, bo + k * kBK, n0);
                    }
                    ++issued;
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                    if (!PROMOTE) {
                        k += ao == 0;
                        ao = other - ao;
                    } else if (++k == nk) {
                        k = 0;
                        ++pair;
                    }
                }
            }
            if constexpr (PAIR) *copies = (int)issued;         // (only the last ring's worth matters below)
            if (!ok) {
                // Let every copy already issued land before the CTA can exit (a
                // pair's CTAs settle this together, below).
                for (int i = 0; !PAIR && i < stages && i < issued; ++i) {
                    if (--stage < 0) { stage = stages - 1; phase ^= 1; }
                    mbar_drain_wait(full_bar(stage), phase);
                }
            } else if (PAIR) {
                // Every commit's arrival is in before either CTA can exit.
                for (int i = 0; i < stages; ++i) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1, abort_flag)) break;
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && rank == 0) {
            auto commit = [&](uint32_t bar) {
                if constexpr (PAIR) umma_commit_pair(bar);
                else                umma_commit(bar);
            };
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued_any = false;
            for (int n_item = first; n_item < jobs.items && ok; n_item += step) {
                int i = n_item;
                const GemmParams& p = jobs.job[job_of(i)];
                const int split = i / (p.n_m * p.n_n), chunks = p.nk * p.pairs;
                const int k0 = (int)((long long)chunks * split / p.splits);
                const int k1 = (int)((long long)chunks * (split + 1) / p.splits);
                const bool a_mn = EPI == EPI_OUT && p.a_mn;
                const uint32_t idesc =
                    umma_idesc_f16(BF16, kTileM, jobs.BN) | (a_mn ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
                // A K step of 16 elements: 32 bytes along a K-major row, 16
                // rows of 128 bytes of an MN-major block.
                const uint32_t a_step = a_mn ? 128 : 2, b_step = B_MN ? 128 : 2;
                for (int q0 = k0; q0 < k1 && ok;) {
                    const int q1 = PROMOTE ? min(k1, q0 + jobs.seg) : k1;
                    if (!mbar_wait(acce_bar(acc), acc_phase ^ 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * 256);
                    for (int q = q0; q < q1; ++q) {
                        if (!mbar_wait(full_bar(stage), phase, abort_flag)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a_addr = smem_addr(smem + stage * stage_bytes), b_addr = a_addr + kABytes;
                        const uint64_t a_desc = a_mn ? sw128_mnmajor_desc(a_addr, 8192u) : sw128_kmajor_desc(a_addr);
                        const uint64_t b_desc = B_MN ? sw128_mnmajor_desc(b_addr, 8192u) : sw128_kmajor_desc(b_addr);
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k) {
                            const uint64_t ad = a_desc + (uint64_t)(k * a_step), bd = b_desc + (uint64_t)(k * b_step);
                            const uint32_t add = (q > q0 || k > 0) ? 1u : 0u;
                            if constexpr (PAIR) umma_f16_pair(d_tmem, ad, bd, idesc, add);
                            else                umma_f16(d_tmem, ad, bd, idesc, add);
                        }
                        issued_any = true;
                        commit(empty_bar(stage));
                        if (++stage == stages) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    commit(accf_bar(acc));
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                    q0 = q1;
                }
            }
            if (!ok && issued_any) {
                if constexpr (PAIR) umma_commit_pair_own(drain_bar);
                else                umma_commit(drain_bar);
                mbar_drain_wait(drain_bar, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Groups of four warps share an accumulator's columns; warp q (mod 4)
        // reads TMEM lanes 32 (q mod 4)..: one output row a lane.
        const int ew = warp - 2, group = ew >> 2, quarter = warp & 3;
        uint32_t* stage = epi_stage + ew * (kStageWarpBytes / 4);
        const int nch = jobs.BN / 32, c_lo = nch * group / kGroups, c_hi = nch * (group + 1) / kGroups;
        // An emptied accumulator is reported to the CTA that issues the MMAs.
        auto emptied = [&](int a) {
            if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(acce_bar(a), 0));
            else                mbar_arrive(acce_bar(a));
        };
        int acc = 0, turn = 0;
        uint32_t acc_phase = 0;
        for (int n_item = first; n_item < jobs.items; n_item += step) {
            int i = n_item;
            const GemmParams& p = jobs.job[job_of(i)];
            const Item it = item_of(p, i);
            const int row0 = it.m * kTileM + rank * kBM + quarter * 32, row = row0 + lane, n0 = it.n * jobs.BN;
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
            bool lands = true;                                 // EPI_LSE: no wait of this tile ran out
            // PROMOTE: this warp's share of the tile's sums, in registers.
            constexpr int kKept = PROMOTE ? 8 / kGroups : 1;   // 32-column chunks per warp at most
            float sum[kKept][32];
            if constexpr (PROMOTE) {
                const int chunks = p.nk * p.pairs;
                const int k0 = (int)((long long)chunks * it.split / p.splits);
                const int k1 = (int)((long long)chunks * (it.split + 1) / p.splits);
#pragma unroll
                for (int c = 0; c < kKept; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
                bool got = true;
                for (int q0 = k0; q0 < k1; q0 += jobs.seg) {
                    got = __all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag));
                    if (!got) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll
                    for (int c = 0; c < kKept; ++c) {
                        if (c_lo + c < c_hi) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {      // 16 at a time: the sums leave few registers
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
                    if (lane == 0) emptied(acc);
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                }
                if (EPI != EPI_LSE && !got) break;
                lands = got;
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
                    const float base = isinf(m_new) ? 0.f : m_new;
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
                        // 16 columns of a row are one memory sector (of each part).
#pragma unroll
                        for (int j = 0; j < 32; j += 16) {
                            uint32_t u[8];
                            if (!PROMOTE || !BF16 || p.parts < 3) {
#pragma unroll
                                for (int l = 0; l < 8; ++l) u[l] = pack2<BF16>(v[j + 2 * l], v[j + 2 * l + 1]);
                                st_global_v8(dst + j, u);
                                if (p.parts == 2) {            // what the rounding left
#pragma unroll
                                    for (int l = 0; l < 8; ++l) {
                                        float a, b;
                                        unpack2<BF16>(u[l], a, b);
                                        u[l] = pack2<BF16>(rest_of(v[j + 2 * l], a), rest_of(v[j + 2 * l + 1], b));
                                    }
                                    st_global_v8(dst + p.dz_part + j, u);
                                }
                            } else {
                                // Part after part: what a part leaves of v goes on to the next.
#pragma unroll
                                for (int s = 0; s < 3; ++s) {
#pragma unroll
                                    for (int l = 0; l < 8; ++l) {
                                        const float a = part_of(v[j + 2 * l]), b = part_of(v[j + 2 * l + 1]);
                                        u[l] = pack2<true>(a, b);
                                        v[j + 2 * l] = rest_of(v[j + 2 * l], a);
                                        v[j + 2 * l + 1] = rest_of(v[j + 2 * l + 1], b);
                                    }
                                    st_global_v8(dst + (int64_t)s * p.dz_part + j, u);
                                }
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
                if (lane == 0) emptied(acc);
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
            if constexpr (EPI == EPI_LSE) {
                // The groups' pairs of a row become one (two buffers in turn:
                // the next tile's meeting shows that this one's are read).
                float2* meet = reinterpret_cast<float2*>(epi_stage) + (turn & 1) * kGroups * 128;
                ++turn;
                meet[group * 128 + quarter * 32 + lane] = make_float2(m_run, s_run);
                if (!named_bar_and(1, kEpiWarps * 32, lands)) break;
                if (group == 0 && live) {
#pragma unroll
                    for (int g = 1; g < kGroups; ++g) {
                        const float2 o = meet[g * 128 + quarter * 32 + lane];
                        join(m_run, s_run, o.x, o.y);
                    }
                    p.lse_part[(int64_t)it.n * p.M + row] = make_float2(m_run, s_run);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) {
        // Each CTA leaves its state with the other before they meet: after the meeting
        // the other may be gone, and its memory with it.
        if (threadIdx.x == 0) {
            const uint32_t to = cluster_addr(smem_addr(const_cast<int*>(peer)), rank ^ 1);
            st_cluster(to, (uint32_t)*abort_flag);
            st_cluster(to + 4, (uint32_t)*copies);
        }
        __syncwarp();
        cluster_sync();                                    // both CTAs are done with each other's memory
        if (*abort_flag || peer[0]) {
            // A wait ran out.  The two CTAs may have stopped at different fills;
            // the issuing CTA's barriers count both CTAs' bytes.  It adds what
            // the one that is behind never sent, or expects what the one ahead
            // did send, and sees every copy land before either CTA leaves.
            if (rank == 0 && threadIdx.x == 0) {
                const int own = *copies, far = peer[1];
                const int last = own > far ? own : far;
                for (int c = last > stages ? last - stages : 0; c < last; ++c) {
                    const uint32_t bar = full_bar(c % stages);
                    if (c >= far) mbar_complete_tx(bar, (uint32_t)stage_bytes);
                    else if (c >= own) mbar_arrive_expect_tx(bar, (uint32_t)stage_bytes);
                    if (!mbar_drain_wait(bar, (uint32_t)(c / stages) & 1u)) break;
                }
            }
            __syncthreads();
            cluster_sync();
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 512);
        else                tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------ small kernels
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
__device__ __forceinline__ void ce_coef(const float* dloss, const int64_t* target, int n, int vocab, int64_t ignore,
                                        int per_row, int mean, float* coef, float* common) {
    __shared__ float red[32];
    __shared__ float up_s;
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
__device__ __forceinline__ void ce_pack(const T* src, int64_t stride, int64_t rows, int cols, int pitch, int vec,
                                        const int64_t* target, int vocab, int64_t ignore, uint16_t* dst, int64_t block,
                                        int64_t blocks) {
    const int per = pitch / 8;
    const int64_t total = rows * per;
    for (int64_t i = block * blockDim.x + threadIdx.x; i < total; i += blocks * blockDim.x) {
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
            float x[8], q[8][3];
            if (vec && keep && c + 8 <= cols) {
                const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
                x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
                x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = keep && c + j < cols ? to_f32(s[j]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(x[j], q[j]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4*>(d + (int64_t)k * pitch) =
                    make_uint4(pack2<true>(q[0][k], q[1][k]), pack2<true>(q[2][k], q[3][k]),
                               pack2<true>(q[4][k], q[5][k]), pack2<true>(q[6][k], q[7][k]));
        }
    }
}

template <typename T, int PARTS>
__global__ void __launch_bounds__(256) ce_pack_kernel(const T* src, int64_t stride, int64_t rows, int cols, int pitch,
                                                      int vec, uint16_t* dst) {
    pdl_wait();
    ce_pack<T, PARTS>(src, stride, rows, cols, pitch, vec, nullptr, 0, 0, dst, blockIdx.x, gridDim.x);
}

// What the backward pass starts with: block 0 makes coef and common, the others
// copy h.
template <typename T, int PARTS>
__global__ void __launch_bounds__(1024)
ce_prepare_kernel(const T* h, int64_t stride, int64_t rows, int cols, int pitch, int vec, const float* dloss,
                  const int64_t* target, int vocab, int64_t ignore, int per_row, int mean, float* coef, float* common,
                  uint16_t* dst) {
    pdl_wait();
    if (blockIdx.x == 0) ce_coef(dloss, target, (int)rows, vocab, ignore, per_row, mean, coef, common);
    else ce_pack<T, PARTS>(h, stride, rows, cols, pitch, vec, target, vocab, ignore, dst, blockIdx.x - 1, gridDim.x - 1);
}

// out = scale (acc + sum over splits), or acc = that sum unscaled (to_acc).  The
// sums' rows are lds wide (a multiple of 64); four columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) ce_join_kernel(const float* part, int splits, int64_t rows, int cols, int64_t lds,
                                                      float* acc, int add, int to_acc, const float* scale, T* out) {
    pdl_wait();
    const float s = *scale;
    const int per = (cols + 3) / 4;
    const int64_t total = rows * per, pitch = rows * lds;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 4;
        const int64_t at = row * lds + c;
        float4 v = add ? *reinterpret_cast<const float4*>(acc + at) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < splits; ++k) {
            const float4 t = *reinterpret_cast<const float4*>(part + k * pitch + at);
            v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
        }
        if (to_acc) {
            *reinterpret_cast<float4*>(acc + at) = v;
        } else {
            const float f[4] = {v.x * s, v.y * s, v.z * s, v.w * s};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < cols) out[row * cols + c + j] = from_f32<T>(f[j]);
        }
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


// CTA pairs that run at once (SMs pair up within their cluster hardware).
int pair_count();

// One product of a launch, for the estimate; at least `least` splits.
struct Product { int64_t M, N, chunks; bool may_split; int least; };

// Tile width, CTA pairs and K splits of a launch's products by an estimate in SM
// cycles.  A 64-wide chunk takes its MMAs (2 BN cycles) or its operands' way
// from the L2 (measured 75 bytes a cycle and SM: it is what holds single CTAs
// at 78 % of the MMA rate, and any tile narrower than 256), and a fixed cost;
// an item (one tile of one split) adds pipeline fill and its last epilogue;
// items run in turn over the SMs or pairs, the first product's before the
// second's; splits add the write and read of their fp32 sums and one launch.  Up
// to 64 splits are weighed, or the fewest that the product needs.
LaunchPlan plan_gemm(const Product* pr, int n, int step, bool b_mn) {
    LaunchPlan best{256, false, {1, 1}};
    double best_t = -1;
    for (int pair = 0; pair < 2; ++pair) {
        if (pair && pr[0].M <= kBM && (n == 1 || pr[1].M <= kBM)) break;
        const int units = pair ? pair_count() : device_sm_count(), rows = pair ? 2 * kBM : kBM;
        const int down = pair && b_mn ? 2 * step : step;     // half a tile is whole 64-wide boxes
        for (int bn = 256; bn >= (pair ? 128 : 64); bn -= down) {
            if (bn - down >= pr[0].N && bn - down >= (pair ? 128 : 64)) continue;      // wider than the output needs
            const double bytes = kABytes + (pair ? bn / 2 : bn) * kBK * 2;
            const double chunk = (2.0 * bn > bytes / 75.0 ? 2.0 * bn : bytes / 75.0) + 24.0;
            const int least[2] = {pr[0].least, n > 1 ? pr[1].least : 1};
            const int most[2] = {least[0] > 64 ? least[0] : 64, least[1] > 64 ? least[1] : 64};
            for (int s0 = least[0]; s0 <= most[0]; s0 = s0 < 4 ? s0 + 1 : s0 + s0 / 2) {
                if (s0 > least[0] && (!pr[0].may_split || s0 > pr[0].chunks)) break;
                for (int s1 = least[1]; s1 <= most[1]; s1 = s1 < 4 ? s1 + 1 : s1 + s1 / 2) {
                    if (s1 > least[1] && (n == 1 || !pr[1].may_split || s1 > pr[1].chunks)) break;
                    const int s[2] = {s0, s1};
                    int64_t items[2] = {0, 0};
                    double each[2] = {0, 0}, t = 0;
                    for (int j = 0; j < n; ++j) {
                        items[j] = ceil_div(pr[j].M, rows) * ceil_div(pr[j].N, bn) * s[j];
                        each[j] = (double)ceil_div(pr[j].chunks, s[j]) * chunk + 3000.0;
                        if (s[j] > 1) t += 4000.0 + (double)s[j] * pr[j].M * pr[j].N * 8.0 / 3500.0;
                    }
                    const int64_t turns = ceil_div(items[0] + items[1], units), turns0 = ceil_div(items[0], units);
                    t += turns0 * each[0] + (turns - turns0) * each[1];
                    // (A unit with a turn less of the first product may be the longest.)
                    const double other = (turns0 - 1) * each[0] + (turns - turns0 + 1) * each[1];
                    if (n > 1 && items[0] % units && other > turns0 * each[0] + (turns - turns0) * each[1])
                        t += other - (turns0 * each[0] + (turns - turns0) * each[1]);
                    if (best_t < 0 || t < best_t * 0.999) {
                        best_t = t;
                        best = LaunchPlan{bn, pair != 0, {s0, s1}};
                    }
                }
            }
        }
    }
    return best;
}

bool allow_smem(const void* kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) == cudaSuccess;
}

constexpr int kFixedSmem = 1024 + (2 * kMaxRing + 5) * 8 + 24;

cudaError_t launch_clusters(const void* kern, int grid, int threads, int ctas, int smem, cudaStream_t st, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

int pair_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return device_sm_count() / 2;
    if (dev >= 0 && dev < 64 && cached[dev]) return cached[dev];
    const void* kern = reinterpret_cast<const void*>(&ce_gemm_kernel<true, EPI_OUT, false, true>);
    int n = 0;
    if (allow_smem(kern)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(device_sm_count() / 2 * 2));
        cfg.blockDim = dim3(32 * (2 + epi_warps(false)));
        cfg.dynamicSmemBytes = kSmemMost;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
    }
    (void)cudaGetLastError();                              // without a GPU: the default below
    if (n < 1) n = device_sm_count() / 2;
    if (dev >= 0 && dev < 64) cached[dev] = n;
    return n;
}

// Where the logits of a 16-bit dz are promoted.  What truncation takes from z, which
// grows with z and the hidden size, is missing from p = exp(z - lse) as a factor,
// while lse comes from the forward pass's promoted sums: all-positive logits of 2.9 on
// average lowered dh and dw by 6e-5 at 4096 features, 2.9e-4 at 16384.  One segment of
// the forward pass is as exact here without; beyond it fp16 promotes, and bf16, whose
// own rounding is eight times coarser, from eight times that on.  The promoted form
// costs z 3 to 8 % (bf16 8192 x 2048 x 131072 2.70 and 2.91 ms, fp16 4096 x 4096 x
// 32768 0.86 and 0.84 ms, 2000 x 520 x 30001 as one segment 0.09 ms).
bool promote_z(bool bf16, int nk) { return nk > (bf16 ? 128 : 16); }

template <int EPI, bool PAIR> const void* gemm_kernel(bool bf16, bool promote) {
    if constexpr (EPI == EPI_LSE) {
        return bf16 ? reinterpret_cast<const void*>(&ce_gemm_kernel<true, EPI, true, PAIR>)
                    : reinterpret_cast<const void*>(&ce_gemm_kernel<false, EPI, true, PAIR>);
    } else {
        if (promote && bf16) return reinterpret_cast<const void*>(&ce_gemm_kernel<true, EPI, true, PAIR>);
        if constexpr (EPI == EPI_DZ)
            if (promote) return reinterpret_cast<const void*>(&ce_gemm_kernel<false, EPI, true, PAIR>);
        return bf16 ? reinterpret_cast<const void*>(&ce_gemm_kernel<true, EPI, false, PAIR>)
                    : reinterpret_cast<const void*>(&ce_gemm_kernel<false, EPI, false, PAIR>);
    }
}

template <int EPI>
conv2d_status launch_gemm(bool bf16, const LaunchPlan& g, const GemmMaps& maps, GemmJobs& jobs, int n, cudaStream_t st) {
    const bool f32 = jobs.job[0].pairs > 2, promote = f32 || EPI == EPI_LSE || (EPI == EPI_DZ && promote_z(bf16, jobs.job[0].nk));
    const void* kern = g.pair ? gemm_kernel<EPI, true>(bf16, promote) : gemm_kernel<EPI, false>(bf16, promote);
    if (!allow_smem(kern)) return CONV2D_ERR_CUDA;
    const int ctas = g.pair ? 2 : 1;
    jobs.BN = g.BN;
    // Promoted sums: the shortest segment where the tensor cores wait for
    // memory anyway (few rows).  Emptying an accumulator takes about 1.2 us,
    // longer than four chunks: large products of fp32 operands take six (dh
    // of 1000 x 768 x 20011 is 7e-7 off), losses of 16-bit operands sixteen (5e-7).
    jobs.seg = jobs.job[0].M <= 2 * kBM ? 4 : f32 ? 6 : 16;
    jobs.epi_bytes = EPI == EPI_LSE ? 2 * epi_warps(true) / 4 * 128 * (int)sizeof(float2) : 0;
    jobs.items0 = jobs.items = 0;
    for (int j = 0; j < n; ++j) {
        GemmParams& p = jobs.job[j];
        p.n_m = (int)ceil_div(p.M, ctas * kBM);
        p.n_n = (int)ceil_div(p.N, g.BN);
        // Row tiles whose A (read again for every column tile) stays in the L2 beside the streams.
        const int64_t a_tile = (int64_t)ctas * kBM * p.nk * kBK * 2 * (p.pairs > 2 ? 3 : p.pairs);
        const int64_t rows = (24 << 20) / a_tile;
        p.group = (int)(rows < 1 ? 1 : (rows > p.n_m ? p.n_m : rows));
        const int64_t items = (int64_t)p.n_m * p.n_n * p.splits;
        if (jobs.items + items > 0x7fffffffLL) return CONV2D_ERR_UNSUPPORTED;
        jobs.items += (int)items;
        if (j == 0) jobs.items0 = (int)items;
        // Rows that cannot take 16-byte stores, and ragged last columns, go through shared memory.
        if (EPI == EPI_OUT && p.splits == 1 && !p.to_acc && (!p.out_vec || p.N % 32 != 0))
            jobs.epi_bytes = epi_warps(promote) * kStageWarpBytes;
    }
    const int stage_bytes = kABytes + g.BN / ctas * kBK * 2;
    jobs.stages = (kSmemMost - kFixedSmem - jobs.epi_bytes) / stage_bytes;
    if (jobs.stages > kMaxRing) jobs.stages = kMaxRing;
    const int smem = kFixedSmem + jobs.epi_bytes + jobs.stages * stage_bytes;
    const int units = g.pair ? pair_count() : device_sm_count();
    const int grid = (jobs.items < units ? jobs.items : units) * ctas;
    void* args[2] = {const_cast<GemmMaps*>(&maps), &jobs};
    return launch_clusters(kern, grid, 32 * (2 + epi_warps(promote)), ctas, smem, st, args) == cudaSuccess
               ? CONV2D_OK
               : CONV2D_ERR_CUDA;
}

void take(size_t& at, size_t& off, size_t bytes) {
    off = at;
    at += align_up(bytes, 1024);
}

CePlan plan_ce(const linear_ce_desc& d, bool backward) {
    CePlan c{};
    size_t at = 0;
    c.few = linear_ce_is_few(d, backward);
    if (c.few) {
        if (!backward) {
            take(at, c.part, (size_t)d.tokens * linear_ce_few_blocks(d) * sizeof(float2));
            take(at, c.z_target, (size_t)d.tokens * 4);
            take(at, c.row_loss, (size_t)d.tokens * 4);
        } else {
            take(at, c.dz, (size_t)linear_ce_few_dz(d) * 4);
            take(at, c.sums_h, (size_t)linear_ce_few_sums(d) * 4);
        }
        c.total = at + 1024;
        return c;
    }
    const bool f32 = d.dtype == CONV2D_F32;
    c.bf16 = d.dtype != CONV2D_F16;
    c.parts = f32 ? 3 : 1;
    c.pairs = f32 ? 6 : 1;
    // With few rows the rounding of dz to 16 bits does not average out (one large
    // element per row: dw of 31 fp16 tokens was off by 3.1e-4, its own rounding is
    // 2.1e-4): it then keeps what the rounding leaves as a second part.  Backward
    // with one part and with two, bf16: 64 x 4096 x 65536 329 and 369 us, 256 x 1024
    // x 32000 94 and 110 us, 256 x 4096 x 65536 460 and 561 us.
    c.dz_parts = f32 ? 3 : d.dz_parts ? d.dz_parts : d.tokens <= 2 * kBM ? 2 : 1;
    c.out_pairs = f32 ? 6 : c.dz_parts;
    c.pack_w = f32 || d.ws % 8 != 0;
    // The backward pass always copies h: ignored rows must be zero in dw's product.
    c.pack_h = backward || f32 || d.hs % 8 != 0;
    c.dp = ceil_div(d.hidden, 64) * 64;
    // Pieces: the forward pass needs them only for the packed copy of w.
    const int64_t budget = 256LL << 20;
    int64_t piece = ceil_div(d.vocab, 256) * 256;
    if (backward || c.pack_w) {
        int64_t most = budget;
        if (backward) most = budget / (d.tokens * 2 * c.dz_parts);
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
    const Product z{d.tokens, v, nk * c.pairs, false, 1};
    c.z = plan_gemm(&z, 1, backward ? 64 : 32, false);
    if (!backward) {
        take(at, c.part, (size_t)d.tokens * (size_t)(c.pieces * ceil_div(v, c.z.BN)) * sizeof(float2));
        take(at, c.z_target, (size_t)d.tokens * 4);
        take(at, c.row_loss, (size_t)d.tokens * 4);
    } else {
        const int64_t kh = ceil_div(v, 64) * c.out_pairs, kw = ceil_div(d.tokens, 64) * c.out_pairs;
        // Sums of 16-bit operands stay in tensor memory for this many chunks at most,
        // then go on in fp32.  Terms of one sign lose 6e-9 of their sum with each of
        // them (fp16 8192 x 512 x 65536 in one piece: dh -3.9e-4; unsplit 1024 x 4608 x
        // 100000 -6.3e-4): at most a fifth of the result's own rounding.
        const int64_t most_k = c.bf16 ? 2048 : 256;
        const Product out[2] = {{d.tokens, d.hidden, kh, true, f32 ? 1 : (int)ceil_div(kh, most_k)},
                                {v, d.hidden, kw, true, f32 ? 1 : (int)ceil_div(kw, most_k)}};
        c.out = plan_gemm(out, 2, 64, true);
        take(at, c.coef, (size_t)d.tokens * 4);
        take(at, c.common, 4);
        take(at, c.dz, (size_t)d.tokens * (size_t)piece * 2 * c.dz_parts);
        if (c.pieces > 1) take(at, c.acc, (size_t)d.tokens * c.dp * 4);
        if (c.out.splits[0] > 1) take(at, c.sums_h, (size_t)c.out.splits[0] * d.tokens * c.dp * 4);
        if (c.out.splits[1] > 1) take(at, c.sums_w, (size_t)c.out.splits[1] * v * c.dp * 4);
    }
    if (c.pack_h) take(at, c.hp, (size_t)d.tokens * c.dp * 2 * c.parts);
    if (c.pack_w) take(at, c.wp, (size_t)v * c.dp * 2 * c.parts);
    c.total = at + 1024;           // the workspace may start at any multiple of 16 bytes
    return c;
}

cudaError_t pack(const linear_ce_desc& d, const void* src, int64_t stride, int64_t rows, int64_t dp, void* dst,
                 cudaStream_t st) {
    const int64_t work = ceil_div(rows * (dp / 8), 256);
    const int64_t most = (int64_t)device_sm_count() * 16;
    const dim3 grid((unsigned)(work < most ? work : most)), block(256);
    if (d.dtype == CONV2D_F32)
        return launch_after(ce_pack_kernel<float, 3>, grid, block, 0, st, static_cast<const float*>(src), stride, rows,
                            (int)d.hidden, (int)dp, stride % 4 == 0 && aligned_to(src, 16) ? 1 : 0,
                            static_cast<uint16_t*>(dst));
    const int vec = stride % 8 == 0 && aligned_to(src, 16);
    return launch_after(ce_pack_kernel<__half, 1>, grid, block, 0, st, static_cast<const __half*>(src), stride, rows,
                        (int)d.hidden, (int)dp, vec, static_cast<uint16_t*>(dst));
}

cudaError_t prepare(const linear_ce_desc& d, const CePlan& c, const void* h, const int64_t* target, const float* dloss,
                    float* coef, float* common, void* dst, cudaStream_t st) {
    const int64_t work = ceil_div(d.tokens * (c.dp / 8), 1024);
    const int64_t most = (int64_t)device_sm_count() * 4;
    const dim3 grid((unsigned)(work < most ? work : most) + 1), block(1024);
    const int per_row = d.reduction == HEAD_REDUCE_NONE, mean = d.reduction == HEAD_REDUCE_MEAN;
    if (d.dtype == CONV2D_F32)
        return launch_after(ce_prepare_kernel<float, 3>, grid, block, 0, st, static_cast<const float*>(h), d.hs, d.tokens,
                            (int)d.hidden, (int)c.dp, d.hs % 4 == 0 && aligned_to(h, 16) ? 1 : 0, dloss, target,
                            (int)d.vocab, d.ignore_index, per_row, mean, coef, common, static_cast<uint16_t*>(dst));
    const int vec = d.hs % 8 == 0 && aligned_to(h, 16);
    return launch_after(ce_prepare_kernel<__half, 1>, grid, block, 0, st, static_cast<const __half*>(h), d.hs, d.tokens,
                        (int)d.hidden, (int)c.dp, vec, dloss, target, (int)d.vocab, d.ignore_index, per_row, mean, coef,
                        common, static_cast<uint16_t*>(dst));
}

// h and w as the tensor cores read them: base, columns and row pitch.
struct Operand { const void* base; int64_t cols, pitch; };

conv2d_status gemm_z(const CePlan& c, const linear_ce_desc& d, int epi, const Operand& h, const Operand& w, int64_t rows_w,
                     GemmParams p, cudaStream_t st) {
    p.M = (int)d.tokens;
    p.N = (int)rows_w;
    p.a_mn = 0;
    p.nk = (int)(c.dp / 64);
    p.pairs = c.pairs;
    p.a_part = p.b_part = (int)c.dp;
    p.splits = 1;
    p.vocab = (int)d.vocab;
    p.ignore = d.ignore_index;
    GemmMaps maps;
    if (!make_map(&maps.a[0], h.base, c.bf16, d.tokens, h.cols, h.pitch, kBM) ||
        !make_map(&maps.b[0], w.base, c.bf16, rows_w, w.cols, w.pitch, c.z.BN / (c.z.pair ? 2 : 1)))
        return CONV2D_ERR_CUDA;
    maps.a[1] = maps.a[0];
    maps.b[1] = maps.b[0];
    GemmJobs jobs{};
    jobs.job[0] = p;
    return epi == EPI_LSE ? launch_gemm<EPI_LSE>(c.bf16, c.z, maps, jobs, 1, st)
                          : launch_gemm<EPI_DZ>(c.bf16, c.z, maps, jobs, 1, st);
}

template <typename T> cudaError_t join_splits(const GemmParams& p, const float* sums, void* out, cudaStream_t st) {
    const int64_t work = ceil_div((int64_t)p.M * ceil_div(p.N, 4), 256), most = (int64_t)device_sm_count() * 16;
    return launch_after(ce_join_kernel<T>, dim3((unsigned)(work < most ? work : most)), dim3(256), 0, st, sums, p.splits,
                        (int64_t)p.M, p.N, p.lds, p.acc, p.add, p.to_acc, p.scale, static_cast<T*>(out));
}

// One of the backward products: out = scale (acc + A B^T), split over K when
// planned; A is dz, K-major (for dh) or MN-major (for dw), B is MN-major.
GemmParams out_job(const CePlan& c, const linear_ce_desc& d, int splits, bool a_mn, int64_t M, int64_t K, int64_t b_part,
                   void* out, float* acc, int add, int to_acc, const float* scale, float* sums) {
    GemmParams p{};
    p.M = (int)M;
    p.N = (int)d.hidden;
    p.a_mn = a_mn;
    p.nk = (int)ceil_div(K, 64);
    p.pairs = c.out_pairs;
    p.a_part = (int)c.piece;
    p.b_part = (int)b_part;
    p.splits = splits < p.nk * p.pairs ? splits : p.nk * p.pairs;
    p.ldo = d.hidden;
    p.lds = c.dp;
    p.out_f32 = d.dtype == CONV2D_F32;
    const int64_t row_bytes = d.hidden * (p.out_f32 ? 4 : 2);
    p.out_vec = row_bytes % 32 == 0 && aligned_to(out, 32) ? 2 : row_bytes % 16 == 0 && aligned_to(out, 16) ? 1 : 0;
    p.add = add;
    p.to_acc = to_acc;
    p.acc = acc;
    p.scale = scale;
    p.out = p.splits > 1 ? sums : out;
    return p;
}

cudaError_t join_job(const linear_ce_desc& d, const GemmParams& p, const float* sums, void* out, cudaStream_t st) {
    if (p.splits == 1) return cudaSuccess;
    switch (d.dtype) {
        case CONV2D_F32: return join_splits<float>(p, sums, out, st);
        case CONV2D_F16: return join_splits<__half>(p, sums, out, st);
        default: return join_splits<__nv_bfloat16>(p, sums, out, st);
    }
}

uint8_t* aligned_base(void* ws) {
    return reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(ws), 1024));
}

const void* at_row(const void* base, int64_t row, int64_t stride, size_t e) {
    return static_cast<const uint8_t*>(base) + (size_t)(row * stride) * e;
}

}  // namespace

void linear_ce_plan(linear_ce_desc& d) {
    d.fwd = d.bwd = CePlan{};
    if (d.tokens == 0) return;
    d.sms = device_sm_count();
    d.fwd = plan_ce(d, false);
    d.bwd = plan_ce(d, true);
}

conv2d_status launch_linear_ce_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                                   float* loss, float* lse, void* ws, cudaStream_t st) {
    const CePlan& c = d.fwd;
    uint8_t* base = aligned_base(ws);
    const size_t e = elem_bytes(d.dtype);
    GemmParams p{};
    p.target = target;
    p.z_target = reinterpret_cast<float*>(base + c.z_target);
    float2* part = reinterpret_cast<float2*>(base + c.part);
    int tiles = 0;
    if (c.few) {
        if (launch_ce_few_fwd(d, h, w, target, part, p.z_target, st) != cudaSuccess) return CONV2D_ERR_CUDA;
        tiles = linear_ce_few_blocks(d);
    } else {
        Operand ho{h, d.hidden, d.hs};
        if (c.pack_h) {
            if (pack(d, h, d.hs, d.tokens, c.dp, base + c.hp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
            ho = Operand{base + c.hp, c.dp * c.parts, c.dp * c.parts};
        }
        for (int64_t v0 = 0; v0 < d.vocab; v0 += c.piece) {
            const int64_t rows = d.vocab - v0 < c.piece ? d.vocab - v0 : c.piece;
            Operand wo{at_row(w, v0, d.ws, e), d.hidden, d.ws};
            if (c.pack_w) {
                if (pack(d, wo.base, d.ws, rows, c.dp, base + c.wp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
                wo = Operand{base + c.wp, c.dp * c.parts, c.dp * c.parts};
            }
            p.col0 = (int)v0;
            p.lse_part = part + (size_t)tiles * d.tokens;
            const conv2d_status s = gemm_z(c, d, EPI_LSE, ho, wo, rows, p, st);
            if (s != CONV2D_OK) return s;
            tiles += (int)ceil_div(rows, c.z.BN);
        }
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
    uint8_t* base = aligned_base(ws);
    const size_t e = elem_bytes(d.dtype);
    float* coef = reinterpret_cast<float*>(base + c.coef);
    float* common = reinterpret_cast<float*>(base + c.common);
    float* acc = c.pieces > 1 ? reinterpret_cast<float*>(base + c.acc) : nullptr;
    float *sums_h = reinterpret_cast<float*>(base + c.sums_h), *sums_w = reinterpret_cast<float*>(base + c.sums_w);
    if (c.few)
        return launch_ce_few_bwd(d, h, w, target, lse, dloss, dh, dw, reinterpret_cast<float*>(base + c.dz), sums_h, st) ==
                       cudaSuccess
                   ? CONV2D_OK
                   : CONV2D_ERR_CUDA;
    if (prepare(d, c, h, target, dloss, coef, common, base + c.hp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
    const Operand ho{base + c.hp, c.dp * c.parts, c.dp * c.parts};
    GemmParams p{};
    p.target = target;
    p.lse = lse;
    p.coef = coef;
    p.dz = base + c.dz;
    p.dz_part = (int)c.piece;
    p.parts = c.dz_parts;
    for (int64_t v0 = 0; v0 < d.vocab; v0 += c.piece) {
        const int64_t rows = d.vocab - v0 < c.piece ? d.vocab - v0 : c.piece;
        const bool first = v0 == 0, last = v0 + rows >= d.vocab;
        Operand wo{at_row(w, v0, d.ws, e), d.hidden, d.ws};
        if (c.pack_w) {
            if (pack(d, wo.base, d.ws, rows, c.dp, base + c.wp, st) != cudaSuccess) return CONV2D_ERR_CUDA;
            wo = Operand{base + c.wp, c.dp * c.parts, c.dp * c.parts};
        }
        p.col0 = (int)v0;
        conv2d_status s = gemm_z(c, d, EPI_DZ, ho, wo, rows, p, st);
        if (s != CONV2D_OK) return s;
        // dh and dw of the piece in one launch.
        const int64_t dz_pitch = c.piece * c.dz_parts;
        GemmMaps maps;
        GemmJobs jobs{};
        int n = 0;
        void* dw_out = dw ? static_cast<uint8_t*>(dw) + (size_t)v0 * d.hidden * e : nullptr;
        if (dh) {
            if (!make_map(&maps.a[n], p.dz, c.bf16, d.tokens, dz_pitch, dz_pitch, kBM) ||
                !make_map(&maps.b[n], wo.base, c.bf16, rows, wo.cols, wo.pitch, 64))
                return CONV2D_ERR_CUDA;
            jobs.job[n++] = out_job(c, d, c.out.splits[0], false, d.tokens, rows, c.dp, dh, acc, !first, !last, common,
                                    sums_h);
        }
        if (dw) {
            if (!make_map(&maps.a[n], p.dz, c.bf16, d.tokens, dz_pitch, dz_pitch, 64) ||
                !make_map(&maps.b[n], ho.base, c.bf16, d.tokens, ho.cols, ho.pitch, 64))
                return CONV2D_ERR_CUDA;
            jobs.job[n++] = out_job(c, d, c.out.splits[1], true, rows, d.tokens, c.dp, dw_out, nullptr, 0, 0, common,
                                    sums_w);
        }
        if (n == 1) { maps.a[1] = maps.a[0]; maps.b[1] = maps.b[0]; }
        s = launch_gemm<EPI_OUT>(c.bf16, c.out, maps, jobs, n, st);
        if (s != CONV2D_OK) return s;
        if (dh && join_job(d, jobs.job[0], sums_h, dh, st) != cudaSuccess) return CONV2D_ERR_CUDA;
        if (dw && join_job(d, jobs.job[n - 1], sums_w, dw_out, st) != cudaSuccess) return CONV2D_ERR_CUDA;
    }
    return CONV2D_OK;
}

cudaError_t status_word_ce(void** p) { return unit_status_word(p); }
cudaError_t wait_limit_set_ce(cudaStream_t st, uint64_t ns) { return unit_wait_limit_set(st, ns); }

}  // namespace conv2d_gb300
