// Host-side plans of the training-head operators (include/head.h), shared by
// head_api.cu and the kernels' translation units (not public).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/head.h"
#include "internal.h"

struct layernorm_desc {
    int64_t rows, cols;
    conv2d_dtype dtype, param;
    float eps;
    int64_t xs, ys;      // row strides of x, dx and of y, dy (elements)
    int64_t pixels;      // > 0: x and dx are [rows / pixels][cols][pixels]
};

struct dropout_desc {
    int64_t rows, cols;
    conv2d_dtype dtype;
    double p;
    int64_t xs, rs, ys;  // row strides of x and dx, residual, y and dy
};

namespace conv2d_gb300 {

// Tile width, CTA pairs and K splits of a launch's products (linear_ce.cu, plan_gemm).
struct LaunchPlan { int BN; bool pair; int splits[2]; };

// Sizes and workspace offsets of one pass of the linear cross entropy.
struct CePlan {
    bool few;                      // few tokens: linear_ce_few.cu
    bool bf16, pack_w, pack_h;
    int parts, pairs;              // bf16 parts per value (1, or 3 for fp32) and their products (1 or 6)
    int dz_parts, out_pairs;       // the same for dz and the products that read it (16 bits, few rows: 2 and 2)
    int64_t dp;                    // packed row pitch of one part
    int64_t piece, pieces;         // vocabulary rows per piece
    LaunchPlan z, out;             // the logits; dh and dw together
    size_t part, z_target, row_loss, coef, common, hp, wp, dz, acc, sums_h, sums_w, total;
};

}  // namespace conv2d_gb300

struct linear_ce_desc {
    int64_t tokens, hidden, vocab;
    conv2d_dtype dtype;
    head_reduction reduction;
    int64_t ignore_index;
    int64_t hs, ws;      // row strides of h and w
    int64_t piece;       // vocabulary rows per backward piece; 0 = automatic
    int dz_parts;        // 16-bit parts of dz: 1, 2; 0 = automatic
    int sms;             // of the device that the plans are for: the few-token kernels' blocks and shares
    conv2d_gb300::CePlan fwd, bwd;
};

namespace conv2d_gb300 {

inline size_t elem_bytes(conv2d_dtype t) { return t == CONV2D_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// layernorm.cu
cudaError_t launch_layernorm_fwd(const layernorm_desc& d, const void* x, const void* gamma, const void* beta, void* y,
                                 float* mean, float* rstd, cudaStream_t st);
size_t layernorm_bwd_workspace(const layernorm_desc& d);
cudaError_t launch_layernorm_bwd(const layernorm_desc& d, const void* dy, const void* x, const void* gamma,
                                 const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* ws,
                                 cudaStream_t st);

// The last step of both backward forms: parts x [2][cols] sums added in order.
cudaError_t launch_layernorm_params(const float* part, int parts, const layernorm_desc& d, void* dgamma, void* dbeta,
                                    cudaStream_t st);

// layernorm_planes.cu: x and dx channels-first
cudaError_t launch_layernorm_planes_fwd(const layernorm_desc& d, const void* x, const void* gamma, const void* beta,
                                        void* y, float* mean, float* rstd, cudaStream_t st);
size_t layernorm_planes_bwd_workspace(const layernorm_desc& d);
cudaError_t launch_layernorm_planes_bwd(const layernorm_desc& d, const void* dy, const void* x, const void* gamma,
                                        const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                                        void* ws, cudaStream_t st);

// dropout.cu: y = residual + keep x scale (residual may be null)
cudaError_t launch_dropout(const dropout_desc& d, const void* x, int64_t xs, const void* residual, int64_t rs, void* y,
                           int64_t ys, uint64_t seed, uint64_t offset, cudaStream_t st);

// linear_ce.cu
void linear_ce_plan(linear_ce_desc& d);      // sets fwd and bwd from the rest
conv2d_status launch_linear_ce_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                                   float* loss, float* lse, void* ws, cudaStream_t st);
conv2d_status launch_linear_ce_bwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                                   const float* lse, const float* dloss, void* dh, void* dw, void* ws,
                                   cudaStream_t st);

// linear_ce_few.cu: few tokens, on the CUDA cores
bool linear_ce_is_few(const linear_ce_desc& d, bool backward);
inline int linear_ce_few_blocks(const linear_ce_desc& d) { return d.sms; }   // (max, sum) pairs per token, forward
int64_t linear_ce_few_dz(const linear_ce_desc& d);   // fp32 words of dz and of the partial sums of dh
int64_t linear_ce_few_sums(const linear_ce_desc& d);
cudaError_t launch_ce_few_fwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target, void* part,
                              float* z_target, cudaStream_t st);
cudaError_t launch_ce_few_bwd(const linear_ce_desc& d, const void* h, const void* w, const int64_t* target,
                              const float* lse, const float* dloss, void* dh, void* dw, float* dz, float* sums,
                              cudaStream_t st);

}  // namespace conv2d_gb300
