// The gated feed-forward block, forward and backward, on the 5th-generation tensor
// cores (tcgen05 MMA, accumulators in tensor memory, operands fed by TMA).
//
//   forward    g = x Wg^T and u = x Wu^T share a tile's accumulator, one half
//              each; the epilogue turns them into h = act(g) u in 16 bits, so the
//              pre-activations leave only when the backward pass wants them (saved, in
//              fp32; h is then kept too).  Then y = residual + h Wd^T.
//   backward   dh = dy Wd never leaves either: its epilogue reads the saved g and u
//              and writes dg = dh u act'(g) and du = dh act(g) in 16 bits.
//              Then one launch has all products that are left, the long ones first:
//              dx = [dg du] [Wg; Wu] (one product over both halves of K),
//              dWg = dg^T x, dWu = du^T x, dWd = dy^T h.
//
// All run in one kernel (ffn_gemm_kernel): C[M][N] = sum_k A[m][k] B[n][k] in
// 64-wide K chunks, each operand stored along K (K-major) or along its own rows
// (MN-major: Wd for dh, Wg and Wu for dx, both operands of the weights' gradients),
// so nothing is transposed in memory.  A CTA pair's tile is 256 rows by BN columns, each
// CTA with half of the columns' operand: in the first product one holds Wg's rows, the
// other Wu's.
//
// h, dg and du are rounded to the operands' type: they are the next products'
// operands, and their errors average out over those sums (a result is off by 1.4 times its
// own rounding).  For fp16, whose range gradients leave easily, dg and du are held times a
// power of two that takes the largest of them to [2^10, 2^15) (Held).  g and u are saved in fp32:
// their rounding would pass through act' into every gradient, and the memory is idle
// beside these products.  They lie as the epilogues' lanes, a row each, read them: four columns
// of 32 rows are 512 bytes in a row.
//
// fp32 operands are split into three bf16 parts each and the six products of parts
// that matter are accumulated, the small ones first; tensor memory then holds a few
// chunks' sums at a time, which the epilogue adds in registers, rounded to nearest
// (PROMOTE).  16-bit sums stay in tensor memory, whose truncation costs them a fifth of
// the result's rounding at most (most_chunks), and go on in fp32 after that.
//
// Measured, one launch at a time (SM clock 1.9 GHz; in a loop the large ones run at the power
// limit).  bf16 8192 x 2048 x 8192: h 322 us (1.71 PFLOP/s), y 200 (1.37: 256 x 192 tiles are 3.75 rounds
// of the machine's 76 pairs), dg and du 226 (1.22), the gradients 838 (1.64).  A chunk takes 690
// cycles of a pair of SMs instead of the MMAs' 512: their reads of shared memory and the copies'
// writes together are all that it gives.  50176 x 512 x 1408: 156, 53, 172 and 252 us; h and dg, du are bound
// by memory there (706 MB and 850 MB: 104 and 125 us) and by the epilogue behind few chunks a tile.  What that takes, forward
// passes without `saved`, us: 8192 x 1024 x 4096 151 with gelu, 132 with silu, 129 without an activation, 126 without h's
// stores either; 50176 x 512 x 1408 195, 159 (gelu_tanh 165), 151 and 145.
// What each step brought at 8192 x 2048 x 8192 / 50176 x 512 x 1408: saved values as the lanes read them, dg and du
// 339 to 338 / 330 to 273; the accumulator reported free before the stores (an arrival that orders the
// thread's stores waits for all of them), h 327 to 326 / 190 to 152; saved values through shared memory by asynchronous
// copies and h kept rather than written again, dg and du 338 to 225 / 273 to 174; the long items' remainder evened out,
// gradients 892 to 838 / 265 to 252.  Saved values fetched to the L2 a tile ahead made it slower (366 / 296).
#include <cuda.h>
#include <math.h>

#include <initializer_list>
#include <utility>

#include "gated_ffn_device.cuh"
#include "head_device.cuh"
#include "head_gemm.cuh"
#include "head_internal.h"
#include "ptx.cuh"

namespace conv2d_gb300 {

namespace {

enum Product { GATE = 0, ROWS = 1, DGATE = 2, GRADS = 3 };     // h; y; dg and du; dx and the weights' gradients

// What the scale of fp16's dg and du goes by.  Their largest is wanted in [2^10, 2^15): past 65504 they would be
// infinite, and what is below 2^-24 of 2^10 loses digits to subnormal numbers.  The first launch of
// dg and du guesses from dy alone: their largest is 2^-2 to 2^3 of dy's where the weights keep the size of what passes
// through.  It leaves the largest ones, in fp32 and unscaled, and a second launch does the work again where
// the guess was off, else returns at once.  A step of 777 x 509 x 1371 takes 75 us with that and 71 without, one of 8192 x
// 2048 x 8192 1670 where the guess holds and 1950 where it does not (Wd 64 times as large).
struct Held {
    const uint32_t* dy;      // maxima of |dy|, as bits of fp16 (finite values only), or null: no scale
    const uint32_t* dgu;     // maxima of |dg| and |du|, as bits of fp32 (finite values only), or null: not known yet
    int n_dy, n_dgu;
};

struct FfnJob {
    int M, N;                // valid extents of the result
    int n_m, n_n;            // tiles
    int group;               // row tiles that share each column tile before the next one is taken
    int nk, nk0;             // K chunks of one product of parts; those that read the first B
    int a_mn, a_off;         // A is MN-major; its first column
    int a_part, b_part;      // column offset from one part to the next
    int splits, items;
    int scaled;              // the result is held times the factor of dg and du
    void* out;               // final element type
    float* sums;             // splits > 1: partial sums [split][M][lds]
    int64_t ldo, lds, ldr;
    const void* res;         // added to the result, or null
    int out_vec, res_vec;    // rows take 32-byte (2), 16-byte (1) or no wide accesses (0)
};

// A launch: one product, or all that are left at the end (the items of the first,
// longest one come first, those of the last fill the last wave).
struct FfnJobs {
    FfnJob job[4];
    int n, items;
    int long_items, extra;   // items of the products with the long ones; as many of the others take as long as one of these
    int BN, stages, seg;     // tile width, ring depth; PROMOTE: chunks per accumulation in tensor memory
    int epi_bytes;           // epilogue staging in shared memory (0: none needed)
    int pairs, parts, f32;
    int act;
    int inner, fp;           // columns of h, and its pitch
    uint16_t *h, *dgu;       // GATE [M][parts][fp], DGATE [M][parts][2][fp]
    float* saved;            // [M / 32][2][fp / 4][32][4]: a warp's rows side by side, or null
    Held held;
    uint32_t* largest;       // DGATE: where a CTA leaves its largest |dg| and |du|, or null
    int again;               // DGATE: the second launch
    int ctas;                // of the launch
};
struct FfnMaps { CUtensorMap a[4], b[4], b2; };

// The exponent of that scale, of either sign so that 2^e and 2^-e are normal numbers.  By a whole warp.
__device__ __forceinline__ int held_exponent(const Held& h) {
    if (!h.dy) return 0;
    const auto largest = [](const uint32_t* at, int count) {
        uint32_t top = 0;
        for (int i = threadIdx.x & 31; i < count; i += 32) top = max(top, at[i]);
        return __reduce_max_sync(0xffffffffu, top);
    };
    int e = 0;
    const uint32_t dy = largest(h.dy, h.n_dy);             // (2^-24 .. 2^15, or zero)
    if (dy) e = 12 + 127 - (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)dy))) >> 23);
    if (h.dgu) {
        const uint32_t top = largest(h.dgu, h.n_dgu);
        const int k = (int)(top >> 23) - 127;
        if (top && (k + e < 10 || k + e > 14)) e = min(14 - k, 126);
    }
    return e;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

struct Item { int m, n, split; };
__device__ __forceinline__ Item item_of(const FfnJob& p, int i) {
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

// Sixteen columns of a row in 16 bits (a memory sector), or as three bf16 parts `part` apart.
template <bool BF16, bool PROMOTE>
__device__ __forceinline__ void store16(uint16_t* dst, int part, int parts, float (&v)[16]) {
    uint32_t u[8];
    if (!PROMOTE || !BF16 || parts == 1) {
#pragma unroll
        for (int l = 0; l < 8; ++l) u[l] = pack2<BF16>(v[2 * l], v[2 * l + 1]);
        st_global_v8(dst, u);
    } else {
        // Part after part: what a part leaves of v goes on to the next.
#pragma unroll
        for (int s = 0; s < 3; ++s) {
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const float a = part_of(v[2 * l]), b = part_of(v[2 * l + 1]);
                u[l] = pack2<true>(a, b);
                v[2 * l] = rest_of(v[2 * l], a);
                v[2 * l + 1] = rest_of(v[2 * l + 1], b);
            }
            st_global_v8(dst + (int64_t)s * part, u);
        }
    }
}

template <bool BF16> __device__ __forceinline__ float load_out(const void* p, int f32, int64_t i) {
    if (f32) return static_cast<const float*>(p)[i];
    if (BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
    return to_f32(static_cast<const __half*>(p)[i]);
}

// ------------------------------------------------------------------ epilogue of ROWS and GRADS
// One 32-column chunk of an output row (this lane's) in v.
template <bool BF16>
__device__ __forceinline__ void store_out(const FfnJobs& jobs, const FfnJob& p, float (&v)[32], int row0, int row, int c0,
                                          int split, float scale, uint32_t* stage, int lane) {
    const bool live = row < p.M;
    const int n = p.N - c0;                                // valid columns from c0 on
    if (p.splits > 1) {
        float* dst = p.sums + ((int64_t)split * p.M + row) * p.lds + c0;
        if (!live || c0 >= p.lds) return;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
            st_global_v8(dst + i, w);
        }
        return;
    }
    if (p.scaled) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= scale;
    }
    const int f32 = jobs.f32;
    if (p.out_vec && n >= 32 && (!p.res || p.res_vec)) {
        if (!live) return;
        if (p.res) {
            const int64_t at = (int64_t)row * p.ldr + c0;
            if (f32) {
                const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(p.res) + at);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 t = r[i];
                    v[4 * i] += t.x; v[4 * i + 1] += t.y; v[4 * i + 2] += t.z; v[4 * i + 3] += t.w;
                }
            } else {
                const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.res) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 t = r[i];
                    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, b;
                        unpack2<BF16>(w[j], a, b);
                        v[8 * i + 2 * j] += a;
                        v[8 * i + 2 * j + 1] += b;
                    }
                }
            }
        }
        if (f32) {
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
    // memory, so that a warp's accesses run along a row.
    const int rows = min(32, p.M - row0);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) stage[lane * 17 + i] = __float_as_uint(v[half * 16 + i]);
        __syncwarp();
        const int c = half * 16 + (lane & 15), r0 = lane >> 4;
        // Eight rows' residuals are on their way together.
#pragma unroll 1
        for (int k0 = r0; k0 < 32; k0 += 16) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] = p.res && c < n && k0 + 2 * k < rows
                           ? load_out<BF16>(p.res, f32, (int64_t)(row0 + k0 + 2 * k) * p.ldr + c0 + c) : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c < n && k0 + 2 * k < rows)
                    store_param(p.out, f32, BF16, (int64_t)(row0 + k0 + 2 * k) * p.ldo + c0 + c,
                                f[k] + __uint_as_float(stage[(k0 + 2 * k) * 17 + (lane & 15)]));
            }
        }
    }
}

constexpr int kSavedWarpBytes = 32 * 16 * 2 * 4;           // DGATE, a warp: sixteen columns of g and u of its rows

// Epilogue warps: sixteen where the activation or the adding of segments keeps them busy.
__host__ __device__ constexpr int ffn_epi_warps(int product, bool promote) {
    return epi_warps(promote || product == GATE || product == DGATE);
}

template <bool BF16, int PRODUCT, bool PROMOTE, bool PAIR>
__global__ void __launch_bounds__(32 * (2 + ffn_epi_warps(PRODUCT, PROMOTE)), 1)
ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnJobs jobs) {
    if constexpr (PRODUCT == DGATE && !BF16) {
        if (jobs.again) {
            pdl_wait();
            Held guess = jobs.held;
            guess.dgu = nullptr;
            if (held_exponent(guess) == held_exponent(jobs.held)) return;      // (all CTAs alike)
        }
    }
    constexpr bool B_MN = PRODUCT == DGATE || PRODUCT == GRADS;
    constexpr int kEpiWarps = ffn_epi_warps(PRODUCT, PROMOTE), kGroups = kEpiWarps / 4;
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

    // Items are dealt out in turn; every role walks them alike.  Units that get one fewer of the
    // longer items get `extra` of the others before all take turns again.
    const int unit = blockIdx.x / kCtas, units = gridDim.x / kCtas;
    const int long_items = jobs.long_items, more = long_items % units, in_turn = long_items + jobs.extra * (units - more);
    auto after = [&](int i) {
        if (PRODUCT != GRADS || !jobs.extra || i >= in_turn) return i + units;
        if (i < long_items) {
            if (i + units < long_items) return i + units;
            if (unit >= more) return long_items + unit - more;
        } else if (i + units - more < in_turn) {
            return i + units - more;
        }
        return in_turn + unit;
    };
    const int first = PRODUCT != GRADS || unit < long_items ? unit : after(unit - units);
    auto job_of = [&](int& i) {                            // product of item i, which becomes its number there
        int j = 0;
        if constexpr (PRODUCT == GRADS) {
            while (j + 1 < jobs.n && i >= jobs.job[j].items) i -= jobs.job[j++].items;
        }
        return j;
    };
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            for (int n_item = first; n_item < jobs.items && ok; n_item = after(n_item)) {
                int i = n_item;
                const int j = job_of(i);
                const FfnJob& p = jobs.job[j];
                const CUtensorMap *amap = &maps.a[j], *bmap = &maps.b[j];
                const Item it = item_of(p, i);
                const int chunks = p.nk * jobs.pairs;
                const int k0 = (int)((long long)chunks * it.split / p.splits);
                const int k1 = (int)((long long)chunks * (it.split + 1) / p.splits);
                const int m0 = it.m * kTileM + rank * kBM, n0 = it.n * jobs.BN + rank * bn;
                const int f0 = it.n * (jobs.BN / 2);       // GATE: the tile's first row of both weights
                const int nk = p.nk, a_mn = p.a_mn;
                int pair = k0 / nk, k = k0 - pair * nk;
                for (int q = k0; q < k1; ++q) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1, abort_flag)) { ok = false; break; }
                    // A pair's copies all count on the issuing CTA's barrier.
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), (uint32_t)(kCtas * stage_bytes));
                    const uint32_t bar = PAIR ? cluster_addr(full_bar(stage), 0) : full_bar(stage);
                    const uint32_t a_dst = smem_addr(smem + stage * stage_bytes), b_dst = a_dst + kABytes;
                    const int ao = p.a_off + (PROMOTE ? kPartA[pair] * p.a_part : 0);
                    const int bo = PROMOTE ? kPartB[pair] * p.b_part : 0;
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
                        if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, c0, c1);
                        else                tma_load_2d(dst, map, bar, c0, c1);
                    };
                    if (PRODUCT == GRADS && a_mn) {
#pragma unroll
                        for (int l = 0; l < kBM / 64; ++l) load(a_dst + l * 8192, amap, ao + m0 + 64 * l, k * kBK);
                    } else {
                        load(a_dst, amap, ao + k * kBK, m0);
                    }
                    if constexpr (PRODUCT == GATE) {
                        if constexpr (PAIR) {
                            load(b_dst, rank ? &maps.b2 : bmap, bo + k * kBK, f0);
                        } else {
                            load(b_dst, bmap, bo + k * kBK, f0);
                            load(b_dst + bn / 2 * kBK * 2, &maps.b2, bo + k * kBK, f0);
                        }
                    } else if constexpr (B_MN) {
                        const bool other = PRODUCT == GRADS && k >= p.nk0;
                        const CUtensorMap* map = other ? &maps.b2 : bmap;
                        const int kb = (other ? k - p.nk0 : k) * kBK;
                        for (int l = 0; l < bn / 64; ++l) load(b_dst + l * 8192, map, bo + n0 + 64 * l, kb);
                    } else {
                        load(b_dst, bmap, bo + k * kBK, n0);
                    }
                    ++issued;
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                    if (++k == nk) {
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
            for (int n_item = first; n_item < jobs.items && ok; n_item = after(n_item)) {
                int i = n_item;
                const FfnJob& p = jobs.job[job_of(i)];
                const int split = i / (p.n_m * p.n_n), chunks = p.nk * jobs.pairs;
                const int k0 = (int)((long long)chunks * split / p.splits);
                const int k1 = (int)((long long)chunks * (split + 1) / p.splits);
                const bool a_mn = PRODUCT == GRADS && p.a_mn;
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
        // reads TMEM lanes 32 (q mod 4)..: one output row a lane.  A chunk is 32 columns; GATE:
        // 16 (32 for PROMOTE) of g and the same of u, half a tile further on.
        const int ew = warp - 2, group = ew >> 2, quarter = warp & 3;
        uint32_t* stage = epi_stage + ew * ((PRODUCT == DGATE ? kSavedWarpBytes : kStageWarpBytes) / 4);
        constexpr int kUnit = PRODUCT == GATE && !PROMOTE ? 16 : 32;
        const int nch = jobs.BN / kUnit / (PRODUCT == GATE ? 2 : 1), c_lo = nch * group / kGroups, c_hi = nch * (group + 1) / kGroups;
        const int u_col = jobs.BN / 2;
        float up = 1.f, down = 1.f;
        if constexpr (PRODUCT == DGATE && !BF16) up = power_of_two(held_exponent(jobs.held));
        if constexpr (PRODUCT == GRADS && !BF16) down = power_of_two(-held_exponent(jobs.held));
        float largest = 0.f;                               // DGATE, fp16: of this lane's |dg| and |du|, scaled
        // An accumulator that this warp has read is reported to the CTA that issues the MMAs.
        auto emptied = [&](int a) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster_read(cluster_addr(acce_bar(a), 0));
                else                mbar_arrive(acce_bar(a));
            }
        };
        // DGATE: what is saved for the next sixteen columns (part e of chunk c of an item, or of the
        // warp's next item) is on its way to shared memory while these are worked on, every lane's own
        // values in its own places.
        const uint32_t saved_to = smem_addr(stage) + lane * 16;
        auto fetch_saved = [&](int n_item, int c, int e) {
            if (c == c_hi) {
                c = c_lo;
                n_item = after(n_item);
            }
            if (n_item < jobs.items && c_lo < c_hi) {
                const Item it = item_of(jobs.job[0], n_item);
                const int row0 = it.m * kTileM + rank * kBM + quarter * 32, c0 = it.n * jobs.BN + c * 32 + e * 16;
                if (row0 + lane < jobs.job[0].M && c0 < jobs.fp) {
                    const float* at = jobs.saved + (int64_t)(row0 / 32) * 64 * jobs.fp + (int64_t)c0 * 32 + lane * 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        copy_async<16>(saved_to + k * 512, at + k * 128);
                        copy_async<16>(saved_to + 2048 + k * 512, at + (int64_t)jobs.fp * 32 + k * 128);
                    }
                }
            }
            copy_async_commit();
        };
        auto take_saved = [&](float (&w)[16], float (&q)[16]) {
            copy_async_wait<0>();
            const float4* at = reinterpret_cast<const float4*>(stage);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 g = at[k * 32 + lane], u = at[128 + k * 32 + lane];
                q[4 * k] = g.x; q[4 * k + 1] = g.y; q[4 * k + 2] = g.z; q[4 * k + 3] = g.w;
                w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
            }
        };
        if constexpr (PRODUCT == DGATE) fetch_saved(first, c_lo, 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int n_item = first; n_item < jobs.items; n_item = after(n_item)) {
            int i = n_item;
            const FfnJob& p = jobs.job[job_of(i)];
            const Item it = item_of(p, i);
            const int row0 = it.m * kTileM + rank * kBM + quarter * 32, row = row0 + lane;
            const int n0 = it.n * (PRODUCT == GATE ? jobs.BN / 2 : jobs.BN);
            const bool live = row < p.M;
            // Sixteen columns from c0 on of what is saved: of g, and jobs.fp * 32 further on of u.
            auto saved_at = [&](int c0) {
                return jobs.saved + (int64_t)(row0 / 32) * 64 * jobs.fp + (int64_t)c0 * 32 + lane * 4;
            };
            // Sixteen columns from c0 on of h, or of dg and du: v is g or dh, w is u, q is g (DGATE).
            auto half_chunk = [&](int c0, float (&v)[16], float (&w)[16], float (&q)[16]) {
                if (!live || c0 >= jobs.fp) return;
                const int n = jobs.inner - c0;             // the pitch's last columns are zero
                if constexpr (PRODUCT == GATE) {
                    if (jobs.saved) {
                        float* at = saved_at(c0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            *reinterpret_cast<float4*>(at + k * 128) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                            *reinterpret_cast<float4*>(at + (int64_t)jobs.fp * 32 + k * 128) =
                                make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        }
                    }
                    activated_all<!PROMOTE>(jobs.act, v, [&](int j, float a) { w[j] = j < n ? a * w[j] : 0.f; });
                    store16<BF16, PROMOTE>(jobs.h + (int64_t)row * jobs.parts * jobs.fp + c0, jobs.fp, jobs.parts, w);
                } else {
                    activate_all<!PROMOTE>(jobs.act, q, [&](int j, float a, float slope) {
                        const float d = v[j] * up, u = w[j];
                        v[j] = j < n ? d * u * slope : 0.f;
                        w[j] = j < n ? d * a : 0.f;
                    });
                    if constexpr (!BF16) {
                        if (jobs.largest) {
                            float top = 0.f;
#pragma unroll
                            for (int j = 0; j < 16; ++j) top = fmaxf(top, fmaxf(fabsf(v[j]), fabsf(w[j])));
                            if (isinf(top)) {              // (a NaN is passed over)
                                top = 0.f;
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    if (!isinf(v[j])) top = fmaxf(top, fabsf(v[j]));
                                    if (!isinf(w[j])) top = fmaxf(top, fabsf(w[j]));
                                }
                            }
                            largest = fmaxf(largest, top);
                        }
                    }
                    uint16_t* dst = jobs.dgu + (int64_t)row * jobs.parts * 2 * jobs.fp + c0;
                    store16<BF16, PROMOTE>(dst, 2 * jobs.fp, jobs.parts, v);
                    store16<BF16, PROMOTE>(dst + jobs.fp, 2 * jobs.fp, jobs.parts, w);
                }
            };
            if constexpr (PROMOTE) {
                // This warp's share of the tile's sums, in registers: two chunks, or one of g and one of u (one of dh, whose
                // tiles are 128 columns at most: the activation needs the registers).
                constexpr int kKept = PRODUCT == DGATE ? 1 : 2;
                float sum[kKept][32];
                const int col[2] = {c_lo * 32, PRODUCT == GATE ? u_col + c_lo * 32 : c_lo * 32 + 32};
                const bool has[2] = {c_lo < c_hi, PRODUCT == GATE ? c_lo < c_hi : c_lo + 1 < c_hi};
                const int chunks = p.nk * jobs.pairs;
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
                        if (has[c]) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {      // 16 at a time: the sums leave few registers
                                uint32_t u[16];
                                tmem_ld_32x32b_x16(t_row + col[c] + e * 16, u);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) sum[c][e * 16 + j] += __uint_as_float(u[j]);
                            }
                        }
                    }
                    emptied(acc);
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                }
                if (!got) break;
#pragma unroll
                for (int c = 0; c < (PRODUCT == ROWS || PRODUCT == GRADS ? 2 : 1); ++c) {
                    if (!has[c]) continue;
                    const int c0 = n0 + (c_lo + c) * 32;
                    if constexpr (PRODUCT == GATE || PRODUCT == DGATE) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v[16], w[16], q[16];
                            if constexpr (PRODUCT == DGATE) {
                                take_saved(w, q);
                                fetch_saved(n_item, c_lo + c + e, e ^ 1);
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                v[j] = sum[c][e * 16 + j];
                                if constexpr (PRODUCT == GATE) w[j] = sum[1][e * 16 + j];
                            }
                            half_chunk(c0 + e * 16, v, w, q);
                        }
                    } else if (p.N > c0) {
                        store_out<BF16>(jobs, p, sum[c], row0, row, c0, it.split, down, stage, lane);
                    }
                }
            } else {
                float v[16], w[16], q[16];
                if (!__all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag))) break;
                tc_fence_after();
                const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    const int c0 = n0 + c * kUnit;
                    if constexpr (PRODUCT == GATE || PRODUCT == DGATE) {
#pragma unroll 1
                        for (int e = 0; e < kUnit / 16; ++e) {
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(t_row + c * kUnit + e * 16, r);
                            if constexpr (PRODUCT == GATE) {
                                uint32_t s[16];
                                tmem_ld_32x32b_x16(t_row + u_col + c * kUnit + e * 16, s);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) w[j] = __uint_as_float(s[j]);
                            } else {
                                take_saved(w, q);
                                tmem_ld_wait();
                                fetch_saved(n_item, c + e, e ^ 1);
                            }
                            if (c + 1 == c_hi && e + 1 == kUnit / 16) emptied(acc);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
                            half_chunk(c0 + e * 16, v, w, q);
                        }
                    } else {
                        uint32_t r[32];
                        float v[32];
                        tmem_ld_32x32b_x32(t_row + c * 32, r);
                        tmem_ld_wait();
                        if (c + 1 == c_hi) emptied(acc);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                        if (p.N > c0) store_out<BF16>(jobs, p, v, row0, row, c0, it.split, down, stage, lane);
                    }
                }
                if (c_lo == c_hi) emptied(acc);
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
        }
        if constexpr (PRODUCT == DGATE) copy_async_wait<0>();
        if constexpr (PRODUCT == DGATE && !BF16) {
            __syncwarp();
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(largest / up));
            if (lane == 0) *stage = top;
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PRODUCT == DGATE && !BF16) {
        if (warp == 0 && jobs.largest) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, lane < kEpiWarps ? epi_stage[lane * (kSavedWarpBytes / 4)] : 0u);
            if (lane == 0) jobs.largest[blockIdx.x] = top;
        }
    }
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
// Up to four matrices in the layout that the tensor cores read, one a blockIdx.y.
struct PackJob { const void* src; int64_t stride, rows; int cols, pitch, vec; uint16_t* dst; };
struct PackJobs { PackJob job[4]; };
template <typename T, int PARTS> __global__ void __launch_bounds__(256) ffn_pack_kernel(const PackJobs jobs) {
    pdl_wait();
    const PackJob& p = jobs.job[blockIdx.y];
    pack_parts<T, PARTS>(static_cast<const T*>(p.src), p.stride, p.rows, p.cols, p.pitch, p.vec, nullptr, 0, 0, p.dst,
                         blockIdx.x, gridDim.x);
}

// Bits of the largest finite magnitude of fp16 rows, one value a block: a row that is not finite takes no digits from
// the others.
__global__ void __launch_bounds__(1024) ffn_largest_kernel(const uint16_t* x, int64_t stride, int64_t rows, int cols, uint32_t* out) {
    __shared__ uint32_t red[32];
    pdl_wait();
    uint32_t top = 0;
    const auto add = [&](uint32_t bits) { top = max(top, bits < 0x7c00u ? bits : 0u); };
    const int per = (cols + 7) / 8;
    const bool vec = stride % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 1024) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        const uint16_t* s = x + row * stride + c;
        if (vec && c + 8 <= cols) {
            const uint4 v = *reinterpret_cast<const uint4*>(s);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                add(w[j] & 0x7fffu);
                add(w[j] >> 16 & 0x7fffu);
            }
        } else {
            for (int j = 0; j < 8 && c + j < cols; ++j) add((uint32_t)s[j] & 0x7fffu);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = __reduce_max_sync(0xffffffffu, red[threadIdx.x]);
        if (threadIdx.x == 0) out[blockIdx.x] = top;
    }
}

// out = scale * (sum over splits) + res for the results that were split, one a blockIdx.y.  The sums' rows are
// lds wide (a multiple of 64); four columns a thread.
struct JoinJob { const float* part; const void* res; void* out; int64_t rows, lds, ldr, ldo; int splits, cols, scaled; };
struct JoinJobs { JoinJob job[4]; Held held; };
template <typename T> __global__ void __launch_bounds__(256) ffn_join_kernel(const JoinJobs jobs) {
    pdl_wait();
    const JoinJob& p = jobs.job[blockIdx.y];
    const float s = p.scaled ? power_of_two(-held_exponent(jobs.held)) : 1.f;
    const T* res = static_cast<const T*>(p.res);
    T* out = static_cast<T*>(p.out);
    const int per = (p.cols + 3) / 4;
    const int64_t total = p.rows * per, pitch = p.rows * p.lds;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 4;
        const int64_t at = row * p.lds + c;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < p.splits; ++k) {
            const float4 t = *reinterpret_cast<const float4*>(p.part + k * pitch + at);
            v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
        }
        const float f[4] = {v.x * s, v.y * s, v.z * s, v.w * s};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < p.cols)
                out[row * p.ldo + c + j] = from_f32<T>(res ? f[j] + to_f32(res[row * p.ldr + c + j]) : f[j]);
    }
}

// ------------------------------------------------------------------ host side
// 64-wide chunks of 16-bit operands that a sum stays in tensor memory for at most:
// terms of one sign lose a fifth of the result's unit roundoff there (measured for the
// linear cross entropy's products).
int64_t most_chunks(bool bf16) { return bf16 ? 2048 : 256; }

// One product of a launch, for the estimate.
struct Sized { int64_t M, N, chunks; bool may_split; int64_t least; };

// Of products in the order of their items' lengths: how many count as long (the first, and those that are
// nearly so), and how many items of the others take as long as one of these (0: there are none).
template <typename T> int long_products(const T* length, int n, int* extra) {
    int k = 1;
    while (k < n && length[k] * 4 >= length[0] * 3) ++k;
    *extra = k < n ? (int)((double)length[0] / (double)length[k] + 0.5) : 0;
    return k;
}

// Tile width, CTA pairs and K splits of a launch's products by an estimate in SM
// cycles.  A 64-wide chunk takes its MMAs (2 BN cycles) or its operands' way from
// the L2 (75 bytes a cycle and SM), and a fixed cost; an item (one tile of one
// split) adds pipeline fill and its last epilogue; items go to the SMs or pairs in
// turn, so the load of each follows; splits add the write and read of their fp32 sums
// and one launch.  All products are split so that their items are about equally
// long; up to 64 lengths are weighed.
// Splits or none, us: y of 16 x 4096 x 16384 fp16 76 / 123 (the whole call), 64 x 2048 x 8192 bf16 34 / 58, 1000 x 768 x 2048
// fp32 83 / 120, a step of 50176 x 512 x 1408 bf16 650 / 690.  The 3000 cycles of an item and the 4000 of a join are round: half or
// twice of either leaves twelve calls from 16 to 50176 tokens within 1 %, but for one forward pass (5 % more) and one step (3 %
// either way).
FfnTile plan_tiles(const Sized* pr, int n, Product product, bool f32) {
    const bool b_mn = product == DGATE || product == GRADS;
    FfnTile best{256, false, {1, 1, 1, 1}};
    double best_t = -1;
    int64_t most_m = 0, most_n = 0, most_chunks = 0;
    for (int j = 0; j < n; ++j) {
        most_m = pr[j].M > most_m ? pr[j].M : most_m;
        most_n = pr[j].N > most_n ? pr[j].N : most_n;
        most_chunks = pr[j].chunks > most_chunks ? pr[j].chunks : most_chunks;
    }
    const int share = product == GATE ? 2 : 1;             // columns of a tile for one of the result
    for (int pair = 0; pair < 2; ++pair) {
        if (pair && most_m <= kBM) break;
        const int units = pair ? pair_count() : device_sm_count(), rows = pair ? 2 * kBM : kBM;
        // Boxes of whole 64 columns (MN-major), halves of whole chunks of g and of u, half of either for each CTA.
        const int down = b_mn ? (pair ? 128 : 64) : product == GATE && f32 ? 64 : 32;
        const int smallest = pair ? 128 : 64;
        for (int bn = product == DGATE && f32 ? 128 : 256; bn >= smallest; bn -= down) {
            if ((bn - down) / share >= most_n && bn - down >= smallest) continue;      // wider than the output needs
            const double bytes = kABytes + (pair ? bn / 2 : bn) * kBK * 2;
            const double chunk = (2.0 * bn > bytes / 75.0 ? 2.0 * bn : bytes / 75.0) + 24.0;
            for (int s = 1; s <= 64; s = s < 4 ? s + 1 : s + s / 2) {
                const int64_t longest = ceil_div(most_chunks, s);
                if (s > 1 && s > most_chunks) break;
                FfnTile tile{bn, pair != 0, {1, 1, 1, 1}};
                int64_t start[5] = {0, 0, 0, 0, 0}, items[4];
                double each[4] = {0, 0, 0, 0}, extra = 0;
                for (int j = 0; j < n; ++j) {
                    int64_t k = pr[j].may_split ? ceil_div(pr[j].chunks, longest) : 1;
                    if (k < pr[j].least) k = pr[j].least;
                    if (k > pr[j].chunks) k = pr[j].chunks;
                    tile.splits[j] = (int)k;
                    if (k > 1) extra += 4000.0 + (double)k * pr[j].M * pr[j].N * 8.0 / 3500.0;
                    // (Longest items first, as the launch orders them.)
                    const double length = (double)ceil_div(pr[j].chunks, k) * chunk + 3000.0;
                    int at = j;
                    for (; at > 0 && each[at - 1] < length; --at) {
                        each[at] = each[at - 1];
                        items[at] = items[at - 1];
                    }
                    each[at] = length;
                    items[at] = ceil_div(pr[j].M, rows) * ceil_div(pr[j].N * share, bn) * k;
                }
                for (int j = 0; j < n; ++j) start[j + 1] = start[j] + items[j];
                // The unit with the most work is the first one, or the first of those with one long item fewer (see the
                // kernel's order).
                int turns = 0;
                const int k = long_products(each, n, &turns);
                const int64_t all = start[k], more = all % units, total = start[n], in_turn = all + turns * (units - more);
                const double rest = k < n ? each[k] : 0;
                double t = 0;
                for (int64_t u : {(int64_t)0, more}) {
                    const auto count = [&](int64_t from, int64_t to, int64_t by) { return to > from ? (to - from + by - 1) / by : 0; };
                    double load = (double)count(u, all, units) * each[0] + (double)count(in_turn + u, total, units) * rest;
                    if (u >= more) load += (double)count(all + u - more, in_turn < total ? in_turn : total, units - more) * rest;
                    t = load > t ? load : t;
                }
                t += extra;
                if (best_t < 0 || t < best_t * 0.999) {
                    best_t = t;
                    best = tile;
                }
                bool splits = false;
                for (int j = 0; j < n; ++j) splits = splits || pr[j].may_split;
                if (!splits) break;
            }
        }
    }
    return best;
}

template <int PRODUCT, bool PAIR> const void* gemm_kernel(bool bf16, bool promote) {
    if (promote) return reinterpret_cast<const void*>(&ffn_gemm_kernel<true, PRODUCT, true, PAIR>);
    return bf16 ? reinterpret_cast<const void*>(&ffn_gemm_kernel<true, PRODUCT, false, PAIR>)
                : reinterpret_cast<const void*>(&ffn_gemm_kernel<false, PRODUCT, false, PAIR>);
}

// Chunks of a product's items, and about six more that an item costs beside them.
int length_of(const FfnJobs& jobs, const FfnJob& p) { return (int)ceil_div((int64_t)p.nk * jobs.pairs, p.splits) + 6; }

template <int PRODUCT>
conv2d_status launch_gemm(bool bf16, const FfnTile& g, const FfnMaps& maps, FfnJobs& jobs, cudaStream_t st) {
    const bool promote = jobs.pairs > 1;
    const void* kern = g.pair ? gemm_kernel<PRODUCT, true>(bf16, promote) : gemm_kernel<PRODUCT, false>(bf16, promote);
    if (!allow_smem(kern)) return CONV2D_ERR_CUDA;
    const int ctas = g.pair ? 2 : 1;
    jobs.BN = g.BN;
    jobs.epi_bytes = 0;
    jobs.items = 0;
    for (int j = 0; j < jobs.n; ++j) {
        FfnJob& p = jobs.job[j];
        p.n_m = (int)ceil_div(p.M, ctas * kBM);
        p.n_n = (int)ceil_div((int64_t)p.N * (PRODUCT == GATE ? 2 : 1), g.BN);
        // Row tiles whose A (read again for every column tile) stays in the L2 beside the streams.
        const int64_t a_tile = (int64_t)ctas * kBM * p.nk * kBK * 2 * jobs.parts;
        const int64_t rows = (24 << 20) / a_tile;
        p.group = (int)(rows < 1 ? 1 : (rows > p.n_m ? p.n_m : rows));
        const int64_t items = (int64_t)p.n_m * p.n_n * p.splits;
        if (jobs.items + items > 0x7fffffffLL) return CONV2D_ERR_UNSUPPORTED;
        p.items = (int)items;
        jobs.items += (int)items;
        // Rows that cannot take wide accesses, and ragged last columns, go through shared memory.
        if (PRODUCT == DGATE) jobs.epi_bytes = ffn_epi_warps(PRODUCT, promote) * kSavedWarpBytes;
        if ((PRODUCT == ROWS || PRODUCT == GRADS) && p.splits == 1 && (!p.out_vec || (p.res && !p.res_vec) || p.N % 32 != 0))
            jobs.epi_bytes = ffn_epi_warps(PRODUCT, promote) * kStageWarpBytes;
    }
    int length[4];
    for (int j = 0; j < jobs.n; ++j) length[j] = length_of(jobs, jobs.job[j]);
    const int k = long_products(length, jobs.n, &jobs.extra);
    jobs.long_items = 0;
    for (int j = 0; j < k; ++j) jobs.long_items += jobs.job[j].items;
    const int stage_bytes = kABytes + g.BN / ctas * kBK * 2;
    jobs.stages = (kSmemMost - kFixedSmem - jobs.epi_bytes) / stage_bytes;
    if (jobs.stages > kMaxRing) jobs.stages = kMaxRing;
    const int smem = kFixedSmem + jobs.epi_bytes + jobs.stages * stage_bytes;
    const int units = g.pair ? pair_count() : device_sm_count();
    const int grid = (jobs.items < units ? jobs.items : units) * ctas;
    jobs.ctas = grid;
    void* args[2] = {const_cast<FfnMaps*>(&maps), &jobs};
    return launch_clusters(kern, grid, 32 * (2 + ffn_epi_warps(PRODUCT, promote)), ctas, smem, st, args) == cudaSuccess
               ? CONV2D_OK
               : CONV2D_ERR_CUDA;
}

int wide(const void* p, int64_t row_bytes) {
    return row_bytes % 32 == 0 && aligned_to(p, 32) ? 2 : row_bytes % 16 == 0 && aligned_to(p, 16) ? 1 : 0;
}

// ROWS and GRADS: a result of the final type in rows `ldo` apart.
FfnJob out_job(const gated_ffn_desc& d, int64_t M, int64_t N, int64_t nk, int splits, void* out, int64_t ldo, float* sums) {
    FfnJob p{};
    p.M = (int)M;
    p.N = (int)N;
    p.nk = p.nk0 = (int)nk;
    p.splits = splits;
    p.out = out;
    p.ldo = ldo;
    p.lds = ceil_div(N, 64) * 64;
    p.sums = sums;
    p.out_vec = wide(out, ldo * (int64_t)elem_bytes(d.dtype));
    return p;
}

// The results of a launch that were split over K.
cudaError_t join(const gated_ffn_desc& d, const FfnJobs& jobs, cudaStream_t st) {
    JoinJobs joins{};
    joins.held = jobs.held;
    unsigned n = 0;
    int64_t work = 0;
    for (int j = 0; j < jobs.n; ++j) {
        const FfnJob& p = jobs.job[j];
        if (p.splits == 1) continue;
        joins.job[n++] = JoinJob{p.sums, p.res, p.out, p.M, p.lds, p.ldr, p.ldo, p.splits, p.N, p.scaled};
        const int64_t w = ceil_div((int64_t)p.M * ceil_div(p.N, 4), 256);
        work = w > work ? w : work;
    }
    if (!n) return cudaSuccess;
    const int64_t most = (int64_t)device_sm_count() * 16;
    const dim3 grid((unsigned)(work < most ? work : most), n), block(256);
    switch (d.dtype) {
        case CONV2D_F32: return launch_after(ffn_join_kernel<float>, grid, block, 0, st, joins);
        case CONV2D_F16: return launch_after(ffn_join_kernel<__half>, grid, block, 0, st, joins);
        default: return launch_after(ffn_join_kernel<__nv_bfloat16>, grid, block, 0, st, joins);
    }
}

// The operands of a pass as the tensor cores read them, copied where their rows are
// not: x, dy, Wg, Wu, Wd.
struct Operands { Operand x, dy, wg, wu, wd; };

conv2d_status prepare(const gated_ffn_desc& d, const FfnPlan& c, const void* x, const void* dy, const void* wg,
                      const void* wu, const void* wd, uint8_t* base, Operands& o, cudaStream_t st) {
    o.x = Operand{x, d.hidden, d.xs};
    o.dy = Operand{dy, d.hidden, d.ys};
    o.wg = Operand{wg, d.hidden, d.hidden};
    o.wu = Operand{wu, d.hidden, d.hidden};
    o.wd = Operand{wd, d.inner, d.inner};
    PackJobs jobs;
    int n = 0;
    int64_t most = 0;
    const int64_t v = 16 / (int64_t)elem_bytes(d.dtype);
    const auto flush = [&]() -> bool {
        if (!n) return true;
        const int64_t work = ceil_div(most, 256), cap = (int64_t)device_sm_count() * 16;
        const dim3 grid((unsigned)(work < cap ? work : cap), (unsigned)n), block(256);
        n = 0;
        most = 0;
        return (d.dtype == CONV2D_F32 ? launch_after(ffn_pack_kernel<float, 3>, grid, block, 0, st, jobs)
                                      : launch_after(ffn_pack_kernel<__half, 1>, grid, block, 0, st, jobs)) == cudaSuccess;
    };
    const auto pack = [&](bool copied, Operand& m, int64_t rows, int64_t pitch, size_t at) -> bool {
        if (!copied || !m.base) return true;
        uint16_t* dst = reinterpret_cast<uint16_t*>(base + at);
        jobs.job[n++] = PackJob{m.base, m.pitch, rows, (int)m.cols, (int)pitch, m.pitch % v == 0 && aligned_to(m.base, 16), dst};
        if (rows * (pitch / 8) > most) most = rows * (pitch / 8);
        m = Operand{dst, pitch * c.parts, pitch * c.parts};
        return n < 4 || flush();
    };
    if (!pack(c.pack_x, o.x, d.tokens, c.dp, c.xp) || !pack(c.pack_wh, o.wg, d.inner, c.dp, c.wgp) ||
        !pack(c.pack_wh, o.wu, d.inner, c.dp, c.wup) || !pack(c.pack_wd, o.wd, d.hidden, c.fp, c.wdp) ||
        !pack(c.pack_dy, o.dy, d.tokens, c.dp, c.dyp) || !flush())
        return CONV2D_ERR_CUDA;
    return CONV2D_OK;
}

FfnJobs jobs_of(const gated_ffn_desc& d, const FfnPlan& c) {
    FfnJobs jobs{};
    jobs.n = 1;
    jobs.pairs = c.pairs;
    jobs.parts = c.parts;
    jobs.f32 = d.dtype == CONV2D_F32;
    jobs.act = d.act;
    jobs.inner = (int)d.inner;
    jobs.fp = (int)c.fp;
    // (As for the linear cross entropy: the shortest segment where the tensor cores wait for memory
    // anyway, else one that covers the emptying of an accumulator.)
    jobs.seg = d.tokens <= 2 * kBM ? 4 : 6;
    return jobs;
}

}  // namespace

void gated_ffn_plan(gated_ffn_desc& d) {
    d.fwd = d.bwd = FfnPlan{};
    if (d.tokens == 0) return;
    const bool f32 = d.dtype == CONV2D_F32;
    d.sms = device_sm_count();
    for (int pass = 0; pass < 2; ++pass) {
        FfnPlan& c = pass ? d.bwd : d.fwd;
        size_t at = 0;
        c.bf16 = d.dtype != CONV2D_F16;
        c.parts = f32 ? 3 : 1;
        c.pairs = f32 ? 6 : 1;
        c.dp = ceil_div(d.hidden, 64) * 64;
        c.fp = ceil_div(d.inner, 64) * 64;
        c.few = pass == 0 && gated_ffn_is_few(d);
        if (c.few) {
            take(at, c.h, (size_t)gated_ffn_few_words(d) * 4);
            c.total = at + 1024;
            continue;
        }
        c.pack_x = f32 || d.xs % 8 != 0;
        c.pack_wh = f32 || d.hidden % 8 != 0;
        c.pack_wd = f32 || d.inner % 8 != 0;
        c.pack_dy = pass && (f32 || d.ys % 8 != 0);
        const int64_t T = d.tokens, D = d.hidden, F = d.inner, nd = c.dp / 64, nf = c.fp / 64, nt = ceil_div(T, 64);
        const auto least = [&](int64_t chunks) { return f32 ? 1 : ceil_div(chunks, most_chunks(c.bf16)); };
        if (c.pack_x) take(at, c.xp, (size_t)T * c.dp * 2 * c.parts);
        if (c.pack_wh) {
            take(at, c.wgp, (size_t)F * c.dp * 2 * c.parts);
            take(at, c.wup, (size_t)F * c.dp * 2 * c.parts);
        }
        if (c.pack_wd) take(at, c.wdp, (size_t)D * c.fp * 2 * c.parts);
        if (c.pack_dy) take(at, c.dyp, (size_t)T * c.dp * 2 * c.parts);
        if (!pass) {
            take(at, c.h, (size_t)T * c.fp * 2 * c.parts);
            const Sized gate{T, c.fp, nd * c.pairs, false, 1}, rows{T, D, nf * c.pairs, true, least(nf)};
            c.first = plan_tiles(&gate, 1, GATE, f32);
            c.last = plan_tiles(&rows, 1, ROWS, f32);
            if (c.last.splits[0] > 1) take(at, c.sums[0], (size_t)c.last.splits[0] * T * c.dp * 4);
        } else {
            take(at, c.dgu, (size_t)T * 2 * c.fp * 2 * c.parts);
            take(at, c.largest, (size_t)d.sms * 4);
            take(at, c.largest_dgu, (size_t)d.sms * 4);
            const Sized dgate{T, c.fp, nd * c.pairs, false, 1};
            c.first = plan_tiles(&dgate, 1, DGATE, f32);
            const Sized grads[4] = {{T, D, 2 * nf * c.pairs, true, least(2 * nf)},
                                    {F, D, nt * c.pairs, true, least(nt)},
                                    {F, D, nt * c.pairs, true, least(nt)},
                                    {D, F, nt * c.pairs, true, least(nt)}};
            c.last = plan_tiles(grads, 4, GRADS, f32);
            const size_t sums[4] = {(size_t)T * c.dp, (size_t)F * c.dp, (size_t)F * c.dp, (size_t)D * c.fp};
            for (int j = 0; j < 4; ++j)
                if (c.last.splits[j] > 1) take(at, c.sums[j], (size_t)c.last.splits[j] * sums[j] * 4);
        }
        c.total = at + 1024;           // the workspace may start at any multiple of 16 bytes
    }
}

// What is saved: g and u, then h as the products read it.
size_t gated_ffn_saved_bytes(const gated_ffn_desc& d) {
    const int64_t fp = ceil_div(d.inner, 64) * 64;
    return (size_t)ceil_div(d.tokens, 32) * 64 * fp * 4 + (size_t)d.tokens * fp * 2 * (d.dtype == CONV2D_F32 ? 3 : 1);
}
uint16_t* gated_ffn_saved_h(const gated_ffn_desc& d, const float* saved) {
    return reinterpret_cast<uint16_t*>(const_cast<float*>(saved) + ceil_div(d.tokens, 32) * 64 * (ceil_div(d.inner, 64) * 64));
}

conv2d_status launch_gated_ffn_fwd(const gated_ffn_desc& d, const void* x, const void* wg, const void* wu, const void* wd,
                                   const void* residual, void* y, float* saved, void* ws, cudaStream_t st) {
    const FfnPlan& c = d.fwd;
    uint8_t* base = aligned_base(ws);
    if (c.few)
        return launch_gated_ffn_few(d, x, wg, wu, wd, residual, y, saved, reinterpret_cast<float*>(base + c.h), st) ==
                       cudaSuccess
                   ? CONV2D_OK
                   : CONV2D_ERR_CUDA;
    Operands o;
    conv2d_status s = prepare(d, c, x, nullptr, wg, wu, wd, base, o, st);
    if (s != CONV2D_OK) return s;
    const int64_t T = d.tokens, D = d.hidden, F = d.inner;
    FfnMaps maps;
    // h
    FfnJobs jobs = jobs_of(d, c);
    jobs.h = saved ? gated_ffn_saved_h(d, saved) : reinterpret_cast<uint16_t*>(base + c.h);
    jobs.saved = saved;
    FfnJob& p = jobs.job[0];
    p.M = (int)T;
    p.N = (int)c.fp;                                       // h is read in whole chunks: zeros past its columns
    p.nk = p.nk0 = (int)(c.dp / 64);
    p.a_part = p.b_part = (int)c.dp;
    p.splits = 1;
    if (!make_map(&maps.a[0], o.x.base, c.bf16, T, o.x.cols, o.x.pitch, kBM) ||
        !make_map(&maps.b[0], o.wg.base, c.bf16, F, o.wg.cols, o.wg.pitch, c.first.BN / 2) ||
        !make_map(&maps.b2, o.wu.base, c.bf16, F, o.wu.cols, o.wu.pitch, c.first.BN / 2))
        return CONV2D_ERR_CUDA;
    for (int j = 1; j < 4; ++j) { maps.a[j] = maps.a[0]; maps.b[j] = maps.b[0]; }
    s = launch_gemm<GATE>(c.bf16, c.first, maps, jobs, st);
    if (s != CONV2D_OK) return s;
    // y
    FfnJobs last = jobs_of(d, c);
    last.job[0] = out_job(d, T, D, c.fp / 64, c.last.splits[0], y, d.ys, reinterpret_cast<float*>(base + c.sums[0]));
    FfnJob& q = last.job[0];
    q.a_part = q.b_part = (int)c.fp;
    q.res = residual;
    q.ldr = d.ys;
    q.res_vec = residual ? wide(residual, d.ys * (int64_t)elem_bytes(d.dtype)) : 0;
    if (!make_map(&maps.a[0], jobs.h, c.bf16, T, c.fp * c.parts, c.fp * c.parts, kBM) ||
        !make_map(&maps.b[0], o.wd.base, c.bf16, D, o.wd.cols, o.wd.pitch, c.last.BN / (c.last.pair ? 2 : 1)))
        return CONV2D_ERR_CUDA;
    s = launch_gemm<ROWS>(c.bf16, c.last, maps, last, st);
    if (s != CONV2D_OK) return s;
    return join(d, last, st) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

conv2d_status launch_gated_ffn_bwd(const gated_ffn_desc& d, const void* dy, const void* x, const void* wg, const void* wu,
                                   const void* wd, const float* saved, void* dx, void* dwg, void* dwu, void* dwd, void* ws,
                                   cudaStream_t st) {
    const FfnPlan& c = d.bwd;
    uint8_t* base = aligned_base(ws);
    const int64_t T = d.tokens, D = d.hidden, F = d.inner;
    Operands o;
    conv2d_status s = prepare(d, c, x, dy, wg, wu, wd, base, o, st);
    if (s != CONV2D_OK) return s;
    FfnMaps maps;
    FfnJobs jobs = jobs_of(d, c);
    uint16_t* h = gated_ffn_saved_h(d, saved);
    jobs.dgu = reinterpret_cast<uint16_t*>(base + c.dgu);
    jobs.saved = const_cast<float*>(saved);
    if (d.dtype == CONV2D_F16) {
        uint32_t* largest = reinterpret_cast<uint32_t*>(base + c.largest);
        const int64_t work = ceil_div(T * ceil_div(D, 8), 1024);
        jobs.held.n_dy = (int)(work < d.sms ? work : d.sms);
        if (launch_after(ffn_largest_kernel, dim3((unsigned)jobs.held.n_dy), dim3(1024), 0, st,
                         static_cast<const uint16_t*>(dy), d.ys, T, (int)D, largest) != cudaSuccess)
            return CONV2D_ERR_CUDA;
        jobs.held.dy = largest;
        jobs.largest = reinterpret_cast<uint32_t*>(base + c.largest_dgu);
    }
    // dg and du
    FfnJob& p = jobs.job[0];
    p.M = (int)T;
    p.N = (int)c.fp;
    p.nk = p.nk0 = (int)(c.dp / 64);
    p.a_part = (int)c.dp;
    p.b_part = (int)c.fp;
    p.splits = 1;
    if (!make_map(&maps.a[0], o.dy.base, c.bf16, T, o.dy.cols, o.dy.pitch, kBM) ||
        !make_map(&maps.b[0], o.wd.base, c.bf16, D, o.wd.cols, o.wd.pitch, 64))
        return CONV2D_ERR_CUDA;
    for (int j = 1; j < 4; ++j) { maps.a[j] = maps.a[0]; maps.b[j] = maps.b[0]; }
    maps.b2 = maps.b[0];
    s = launch_gemm<DGATE>(c.bf16, c.first, maps, jobs, st);
    if (s != CONV2D_OK) return s;
    if (jobs.largest) {
        jobs.held.dgu = jobs.largest;
        jobs.held.n_dgu = jobs.ctas;
        jobs.largest = nullptr;
        jobs.again = 1;
        s = launch_gemm<DGATE>(c.bf16, c.first, maps, jobs, st);
        if (s != CONV2D_OK) return s;
    }
    // dx and the weights' gradients
    FfnJobs last = jobs_of(d, c);
    last.held = jobs.held;
    last.n = 0;
    float* sums[4];
    for (int j = 0; j < 4; ++j) sums[j] = reinterpret_cast<float*>(base + c.sums[j]);
    const int64_t gu = 2 * c.fp * c.parts, nt = ceil_div(T, 64);
    if (dx) {
        const int j = last.n++;
        FfnJob q = out_job(d, T, D, 2 * c.fp / 64, c.last.splits[0], dx, D, sums[0]);
        q.nk0 = (int)(c.fp / 64);
        q.a_part = (int)(2 * c.fp);
        q.b_part = (int)c.dp;
        q.scaled = 1;
        last.job[j] = q;
        if (!make_map(&maps.a[j], jobs.dgu, c.bf16, T, gu, gu, kBM) ||
            !make_map(&maps.b[j], o.wg.base, c.bf16, F, o.wg.cols, o.wg.pitch, 64) ||
            !make_map(&maps.b2, o.wu.base, c.bf16, F, o.wu.cols, o.wu.pitch, 64))
            return CONV2D_ERR_CUDA;
    }
    for (int k = 0; k < 2; ++k) {
        void* out = k ? dwu : dwg;
        if (!out) continue;
        const int j = last.n++;
        FfnJob q = out_job(d, F, D, nt, c.last.splits[1 + k], out, D, sums[1 + k]);
        q.a_mn = 1;
        q.a_off = (int)(k * c.fp);
        q.a_part = (int)(2 * c.fp);
        q.b_part = (int)c.dp;
        q.scaled = 1;
        last.job[j] = q;
        if (!make_map(&maps.a[j], jobs.dgu, c.bf16, T, gu, gu, 64) ||
            !make_map(&maps.b[j], o.x.base, c.bf16, T, o.x.cols, o.x.pitch, 64))
            return CONV2D_ERR_CUDA;
    }
    if (dwd) {
        const int j = last.n++;
        FfnJob q = out_job(d, D, F, nt, c.last.splits[3], dwd, F, sums[3]);
        q.a_mn = 1;
        q.a_part = (int)c.dp;
        q.b_part = (int)c.fp;
        last.job[j] = q;
        if (!make_map(&maps.a[j], o.dy.base, c.bf16, T, o.dy.cols, o.dy.pitch, 64) ||
            !make_map(&maps.b[j], h, c.bf16, T, c.fp * c.parts, c.fp * c.parts, 64))
            return CONV2D_ERR_CUDA;
    }
    // The products with the longest items first.
    for (int i = 1; i < last.n; ++i)
        for (int j = i; j > 0 && length_of(last, last.job[j - 1]) < length_of(last, last.job[j]); --j) {
            std::swap(last.job[j - 1], last.job[j]);
            std::swap(maps.a[j - 1], maps.a[j]);
            std::swap(maps.b[j - 1], maps.b[j]);
        }
    for (int j = last.n; j < 4; ++j) { maps.a[j] = maps.a[0]; maps.b[j] = maps.b[0]; }
    s = launch_gemm<GRADS>(c.bf16, c.last, maps, last, st);
    if (s != CONV2D_OK) return s;
    return join(d, last, st) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

cudaError_t status_word_ffn(void** p) { return unit_status_word(p); }
cudaError_t wait_limit_set_ffn(cudaStream_t st, uint64_t ns) { return unit_wait_limit_set(st, ns); }

}  // namespace conv2d_gb300
