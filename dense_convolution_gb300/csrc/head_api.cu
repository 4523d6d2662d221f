// C ABI of the training-head operators (include/head.h): descriptors, argument
// checks and workspace sizes.  Host code only; the kernels live in
// layernorm.cu, layernorm_planes.cu, dropout.cu, linear_ce.cu, linear_ce_few.cu,
// gated_ffn.cu, gated_ffn_few.cu and adamw.cu.
#include <math.h>

#include <initializer_list>
#include <new>

#include "head_internal.h"

#define CONV2D_API extern "C" __attribute__((visibility("default")))

using namespace conv2d_gb300;

namespace {

constexpr int64_t kMaxSide = 0x7fffffffLL;
constexpr int64_t kMaxStride = 1LL << 40;
constexpr int64_t kMaxGemmSide = 1LL << 30, kMaxHidden = 1LL << 26;

bool known(conv2d_dtype t) { return t == CONV2D_F32 || t == CONV2D_F16 || t == CONV2D_BF16; }
bool stride_ok(int64_t s, int64_t cols) { return s >= cols && s <= kMaxStride; }
conv2d_status of(cudaError_t e) { return e == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA; }

template <typename D> conv2d_status give(D** out, const D& d) {
    *out = new (std::nothrow) D(d);
    return *out ? CONV2D_OK : CONV2D_ERR_BAD_PARAM;
}

}  // namespace

// ---------------------------------------------------------------- layer norm
CONV2D_API conv2d_status layernorm_desc_create(layernorm_desc_t* out, int64_t rows, int64_t cols, conv2d_dtype dtype,
                                               conv2d_dtype param_dtype, float eps) {
    if (!out) return CONV2D_ERR_NULL_PTR;
    *out = nullptr;
    if (rows < 0 || cols < 1 || rows > kMaxSide || cols > kMaxSide || !known(dtype)) return CONV2D_ERR_BAD_PARAM;
    if (param_dtype != dtype && param_dtype != CONV2D_F32) return CONV2D_ERR_BAD_PARAM;
    if (!(eps >= 0.f) || !isfinite(eps)) return CONV2D_ERR_BAD_PARAM;
    layernorm_desc d{};
    d.rows = rows; d.cols = cols; d.dtype = dtype; d.param = param_dtype; d.eps = eps;
    d.xs = d.ys = cols;
    return give(out, d);
}

CONV2D_API conv2d_status layernorm_desc_set_row_strides(layernorm_desc_t d, int64_t x_stride, int64_t y_stride) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (!stride_ok(x_stride, d->cols) || !stride_ok(y_stride, d->cols)) return CONV2D_ERR_BAD_PARAM;
    if (d->pixels && x_stride != d->cols) return CONV2D_ERR_UNSUPPORTED;
    d->xs = x_stride;
    d->ys = y_stride;
    return CONV2D_OK;
}

CONV2D_API conv2d_status layernorm_desc_set_planes(layernorm_desc_t d, int64_t pixels) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (pixels < 0 || (pixels > 0 && d->rows % pixels != 0)) return CONV2D_ERR_BAD_PARAM;
    if (pixels && (d->xs != d->cols || d->cols > 16384)) return CONV2D_ERR_UNSUPPORTED;
    d->pixels = pixels;
    return CONV2D_OK;
}

CONV2D_API conv2d_status layernorm_desc_destroy(layernorm_desc_t d) {
    delete d;
    return CONV2D_OK;
}

CONV2D_API conv2d_status layernorm_workspace_size(layernorm_desc_t d, size_t* bytes) {
    if (!d || !bytes) return CONV2D_ERR_NULL_PTR;
    *bytes = layernorm_bwd_workspace(*d);
    return CONV2D_OK;
}

CONV2D_API conv2d_status layernorm_fwd(layernorm_desc_t dp, const void* x, const void* gamma, const void* beta,
                                       void* y, float* mean, float* rstd, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const layernorm_desc& d = *dp;
    if (d.rows == 0) return CONV2D_OK;
    if (!x || !y) return CONV2D_ERR_NULL_PTR;
    const size_t e = elem_bytes(d.dtype), pe = elem_bytes(d.param);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(gamma, pe) || !aligned_to(beta, pe) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return CONV2D_ERR_MISALIGNED;
    return of(launch_layernorm_fwd(d, x, gamma, beta, y, mean, rstd, static_cast<cudaStream_t>(stream)));
}

CONV2D_API conv2d_status layernorm_bwd(layernorm_desc_t dp, const void* dy, const void* x, const void* gamma,
                                       const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const layernorm_desc& d = *dp;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t e = elem_bytes(d.dtype), pe = elem_bytes(d.param);
    if (!dx && !dgamma && !dbeta) return CONV2D_OK;
    if (!aligned_to(dgamma, pe) || !aligned_to(dbeta, pe)) return CONV2D_ERR_MISALIGNED;
    if (d.rows == 0) {   // no rows: the sums over rows are zero
        cudaError_t r = cudaSuccess;
        if (dgamma) r = cudaMemsetAsync(dgamma, 0, (size_t)d.cols * pe, st);
        if (r == cudaSuccess && dbeta) r = cudaMemsetAsync(dbeta, 0, (size_t)d.cols * pe, st);
        return of(r);
    }
    const size_t need = layernorm_bwd_workspace(d);
    if (!dy || !x || !mean || !rstd || !workspace) return CONV2D_ERR_NULL_PTR;
    if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(gamma, pe) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(workspace, 16))
        return CONV2D_ERR_MISALIGNED;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    return of(launch_layernorm_bwd(d, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace, st));
}

// ------------------------------------------------------------------- dropout
CONV2D_API conv2d_status dropout_desc_create(dropout_desc_t* out, int64_t rows, int64_t cols, conv2d_dtype dtype,
                                             double p) {
    if (!out) return CONV2D_ERR_NULL_PTR;
    *out = nullptr;
    if (rows < 0 || cols < 1 || rows > kMaxSide || cols > kMaxSide || !known(dtype)) return CONV2D_ERR_BAD_PARAM;
    if (!(p >= 0.0 && p <= 1.0)) return CONV2D_ERR_BAD_PARAM;
    dropout_desc d{};
    d.rows = rows; d.cols = cols; d.dtype = dtype; d.p = p;
    d.xs = d.rs = d.ys = cols;
    return give(out, d);
}

CONV2D_API conv2d_status dropout_desc_set_row_strides(dropout_desc_t d, int64_t x_stride, int64_t residual_stride,
                                                      int64_t y_stride) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (!stride_ok(x_stride, d->cols) || !stride_ok(residual_stride, d->cols) || !stride_ok(y_stride, d->cols))
        return CONV2D_ERR_BAD_PARAM;
    d->xs = x_stride;
    d->rs = residual_stride;
    d->ys = y_stride;
    return CONV2D_OK;
}

CONV2D_API conv2d_status dropout_desc_destroy(dropout_desc_t d) {
    delete d;
    return CONV2D_OK;
}

CONV2D_API conv2d_status dropout_fwd(dropout_desc_t dp, const void* x, const void* residual, void* y, uint64_t seed,
                                     uint64_t offset, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const dropout_desc& d = *dp;
    if (offset >> 63) return CONV2D_ERR_BAD_PARAM;
    if (d.rows == 0) return CONV2D_OK;
    if (!x || !y) return CONV2D_ERR_NULL_PTR;
    const size_t e = elem_bytes(d.dtype);
    if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(y, e)) return CONV2D_ERR_MISALIGNED;
    return of(launch_dropout(d, x, d.xs, residual, d.rs, y, d.ys, seed, offset, static_cast<cudaStream_t>(stream)));
}

CONV2D_API conv2d_status dropout_bwd(dropout_desc_t dp, const void* dy, void* dx, uint64_t seed, uint64_t offset,
                                     void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const dropout_desc& d = *dp;
    if (offset >> 63) return CONV2D_ERR_BAD_PARAM;
    if (d.rows == 0) return CONV2D_OK;
    if (!dy || !dx) return CONV2D_ERR_NULL_PTR;
    const size_t e = elem_bytes(d.dtype);
    if (!aligned_to(dy, e) || !aligned_to(dx, e)) return CONV2D_ERR_MISALIGNED;
    return of(launch_dropout(d, dy, d.ys, nullptr, 0, dx, d.xs, seed, offset, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------- linear cross entropy
CONV2D_API conv2d_status linear_ce_desc_create(linear_ce_desc_t* out, int64_t tokens, int64_t hidden, int64_t vocab,
                                               conv2d_dtype dtype, head_reduction reduction, int64_t ignore_index) {
    if (!out) return CONV2D_ERR_NULL_PTR;
    *out = nullptr;
    if (tokens < 0 || hidden < 1 || vocab < 1 || tokens > kMaxGemmSide || hidden > kMaxHidden ||
        vocab > kMaxGemmSide || !known(dtype))
        return CONV2D_ERR_BAD_PARAM;
    // The kernels number the 128 x 64 tiles of z with 31 bits.
    if (((tokens + 127) / 128) * ((vocab + 63) / 64) > 0x7fffffffLL) return CONV2D_ERR_BAD_PARAM;
    if (reduction != HEAD_REDUCE_NONE && reduction != HEAD_REDUCE_SUM && reduction != HEAD_REDUCE_MEAN)
        return CONV2D_ERR_BAD_PARAM;
    linear_ce_desc d{};
    d.tokens = tokens; d.hidden = hidden; d.vocab = vocab; d.dtype = dtype;
    d.reduction = reduction; d.ignore_index = ignore_index;
    d.hs = d.ws = hidden;
    linear_ce_plan(d);
    return give(out, d);
}

CONV2D_API conv2d_status linear_ce_desc_set_row_strides(linear_ce_desc_t d, int64_t h_stride, int64_t w_stride) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    // A tensor map's row pitch is below 2^40 bytes.
    if (!stride_ok(h_stride, d->hidden) || !stride_ok(w_stride, d->hidden) || h_stride >= kMaxStride / 4 ||
        w_stride >= kMaxStride / 4)
        return CONV2D_ERR_BAD_PARAM;
    d->hs = h_stride;
    d->ws = w_stride;
    linear_ce_plan(*d);
    return CONV2D_OK;
}

CONV2D_API conv2d_status linear_ce_desc_set_piece(linear_ce_desc_t d, int64_t vocab_rows) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (vocab_rows < 0 || vocab_rows > kMaxGemmSide) return CONV2D_ERR_BAD_PARAM;
    d->piece = vocab_rows;
    linear_ce_plan(*d);
    return CONV2D_OK;
}

CONV2D_API conv2d_status linear_ce_desc_set_dz_parts(linear_ce_desc_t d, int parts) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (parts < 0 || parts > 2) return CONV2D_ERR_BAD_PARAM;
    if (parts && d->dtype == CONV2D_F32) return CONV2D_ERR_UNSUPPORTED;
    d->dz_parts = parts;
    linear_ce_plan(*d);
    return CONV2D_OK;
}

CONV2D_API conv2d_status linear_ce_desc_destroy(linear_ce_desc_t d) {
    delete d;
    return CONV2D_OK;
}

CONV2D_API conv2d_status linear_ce_workspace_size(linear_ce_desc_t d, size_t* fwd_bytes, size_t* bwd_bytes) {
    if (!d || (!fwd_bytes && !bwd_bytes)) return CONV2D_ERR_NULL_PTR;
    if (fwd_bytes) *fwd_bytes = d->fwd.total;
    if (bwd_bytes) *bwd_bytes = d->bwd.total;
    return CONV2D_OK;
}

namespace {

// h and w are read in place by tensor copies, which need 16-byte alignment,
// unless they are packed first (or there are few tokens: the interface's rule is
// one for all).
bool ce_operand_ok(const linear_ce_desc& d, const void* p, int64_t stride) {
    const bool packed = d.dtype == CONV2D_F32 || stride % 8 != 0;
    return aligned_to(p, packed ? elem_bytes(d.dtype) : 16);
}

}  // namespace

CONV2D_API conv2d_status linear_ce_fwd(linear_ce_desc_t dp, const void* h, const void* w, const int64_t* target,
                                       float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const linear_ce_desc& d = *dp;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.tokens == 0) {
        if (d.reduction == HEAD_REDUCE_NONE) return CONV2D_OK;
        if (!loss) return CONV2D_ERR_NULL_PTR;
        return of(cudaMemsetAsync(loss, 0, sizeof(float), st));
    }
    if (!h || !w || !target || !loss || !lse || !workspace) return CONV2D_ERR_NULL_PTR;
    if (!ce_operand_ok(d, h, d.hs) || !ce_operand_ok(d, w, d.ws) || !aligned_to(target, 8) || !aligned_to(loss, 4) ||
        !aligned_to(lse, 4) || !aligned_to(workspace, 16))
        return CONV2D_ERR_MISALIGNED;
    if (workspace_bytes < d.fwd.total) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    return launch_linear_ce_fwd(d, h, w, target, loss, lse, workspace, st);
}

CONV2D_API conv2d_status linear_ce_bwd(linear_ce_desc_t dp, const void* h, const void* w, const int64_t* target,
                                       const float* lse, const float* dloss, void* dh, void* dw, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const linear_ce_desc& d = *dp;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!dh && !dw) return CONV2D_OK;
    const size_t e = elem_bytes(d.dtype);
    if (!aligned_to(dh, e) || !aligned_to(dw, e)) return CONV2D_ERR_MISALIGNED;
    if (d.tokens == 0)
        return dw ? of(cudaMemsetAsync(dw, 0, (size_t)d.vocab * d.hidden * e, st)) : CONV2D_OK;
    if (!h || !w || !target || !lse || !dloss || !workspace) return CONV2D_ERR_NULL_PTR;
    if (!ce_operand_ok(d, h, d.hs) || !ce_operand_ok(d, w, d.ws) || !aligned_to(target, 8) || !aligned_to(lse, 4) ||
        !aligned_to(dloss, 4) || !aligned_to(workspace, 16))
        return CONV2D_ERR_MISALIGNED;
    if (workspace_bytes < d.bwd.total) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    return launch_linear_ce_bwd(d, h, w, target, lse, dloss, dh, dw, workspace, st);
}

// ------------------------------------------------- gated feed-forward block
CONV2D_API conv2d_status gated_ffn_desc_create(gated_ffn_desc_t* out, int64_t tokens, int64_t hidden, int64_t inner,
                                               conv2d_dtype dtype, gated_ffn_act act) {
    if (!out) return CONV2D_ERR_NULL_PTR;
    *out = nullptr;
    // (A sum over `hidden` never leaves tensor memory: 16384 is what fp16 takes there.)
    if (tokens < 0 || hidden < 1 || inner < 1 || tokens > kMaxGemmSide || hidden > 16384 || inner > (1LL << 20) ||
        !known(dtype))
        return CONV2D_ERR_BAD_PARAM;
    if (((tokens + 127) / 128) * ((inner + 31) / 32) > 0x7fffffffLL) return CONV2D_ERR_BAD_PARAM;
    if (act != FFN_SILU && act != FFN_GELU && act != FFN_GELU_TANH) return CONV2D_ERR_BAD_PARAM;
    gated_ffn_desc d{};
    d.tokens = tokens; d.hidden = hidden; d.inner = inner; d.dtype = dtype; d.act = act;
    d.xs = d.ys = hidden;
    gated_ffn_plan(d);
    return give(out, d);
}

CONV2D_API conv2d_status gated_ffn_desc_set_row_strides(gated_ffn_desc_t d, int64_t x_stride, int64_t y_stride) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    // A tensor map's row pitch is below 2^40 bytes.
    if (!stride_ok(x_stride, d->hidden) || !stride_ok(y_stride, d->hidden) || x_stride >= kMaxStride / 4 ||
        y_stride >= kMaxStride / 4)
        return CONV2D_ERR_BAD_PARAM;
    d->xs = x_stride;
    d->ys = y_stride;
    gated_ffn_plan(*d);
    return CONV2D_OK;
}

CONV2D_API conv2d_status gated_ffn_desc_destroy(gated_ffn_desc_t d) {
    delete d;
    return CONV2D_OK;
}

CONV2D_API conv2d_status gated_ffn_workspace_size(gated_ffn_desc_t d, size_t* fwd_bytes, size_t* bwd_bytes,
                                                  size_t* saved_bytes) {
    if (!d || (!fwd_bytes && !bwd_bytes && !saved_bytes)) return CONV2D_ERR_NULL_PTR;
    if (fwd_bytes) *fwd_bytes = d->fwd.total;
    if (bwd_bytes) *bwd_bytes = d->bwd.total;
    if (saved_bytes) *saved_bytes = gated_ffn_saved_bytes(*d);
    return CONV2D_OK;
}

namespace {

// Operands are read in place by tensor copies, which need 16-byte alignment, unless they are
// packed first (or there are few tokens: the interface's rule is one for all).
bool ffn_operands_ok(const gated_ffn_desc& d, const void* x, const void* wg, const void* wu, const void* wd) {
    const size_t e = elem_bytes(d.dtype);
    const bool f32 = d.dtype == CONV2D_F32;
    const size_t ax = f32 || d.xs % 8 ? e : 16, ah = f32 || d.hidden % 8 ? e : 16, ad = f32 || d.inner % 8 ? e : 16;
    return aligned_to(x, ax) && aligned_to(wg, ah) && aligned_to(wu, ah) && aligned_to(wd, ad);
}

}  // namespace

CONV2D_API conv2d_status gated_ffn_fwd(gated_ffn_desc_t dp, const void* x, const void* wg, const void* wu,
                                       const void* wd, const void* residual, void* y, float* saved, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const gated_ffn_desc& d = *dp;
    if (d.tokens == 0) return CONV2D_OK;
    if (!x || !wg || !wu || !wd || !y || !workspace) return CONV2D_ERR_NULL_PTR;
    const size_t e = elem_bytes(d.dtype);
    if (!ffn_operands_ok(d, x, wg, wu, wd) || !aligned_to(y, e) || !aligned_to(residual, e) || !aligned_to(saved, 32) ||
        !aligned_to(workspace, 16))
        return CONV2D_ERR_MISALIGNED;
    if (workspace_bytes < d.fwd.total) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    return launch_gated_ffn_fwd(d, x, wg, wu, wd, residual, y, saved, workspace, static_cast<cudaStream_t>(stream));
}

CONV2D_API conv2d_status gated_ffn_bwd(gated_ffn_desc_t dp, const void* dy, const void* x, const void* wg,
                                       const void* wu, const void* wd, const float* saved, void* dx, void* dwg,
                                       void* dwu, void* dwd, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const gated_ffn_desc& d = *dp;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t e = elem_bytes(d.dtype);
    if (!dx && !dwg && !dwu && !dwd) return CONV2D_OK;
    if (!aligned_to(dx, e) || !aligned_to(dwg, e) || !aligned_to(dwu, e) || !aligned_to(dwd, e))
        return CONV2D_ERR_MISALIGNED;
    if (d.tokens == 0) {   // no rows: the sums over rows are zero
        for (void* p : {dwg, dwu, dwd})
            if (p && cudaMemsetAsync(p, 0, (size_t)d.hidden * d.inner * e, st) != cudaSuccess) return CONV2D_ERR_CUDA;
        return CONV2D_OK;
    }
    if (!dy || !x || !wg || !wu || !wd || !saved || !workspace) return CONV2D_ERR_NULL_PTR;
    const size_t ay = d.dtype == CONV2D_F32 || d.ys % 8 ? e : 16;
    if (!ffn_operands_ok(d, x, wg, wu, wd) || !aligned_to(dy, ay) || !aligned_to(saved, 32) || !aligned_to(workspace, 16))
        return CONV2D_ERR_MISALIGNED;
    if (workspace_bytes < d.bwd.total) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    return launch_gated_ffn_bwd(d, dy, x, wg, wu, wd, saved, dx, dwg, dwu, dwd, workspace, st);
}

// --------------------------------------------------------------------- AdamW
CONV2D_API conv2d_status adamw_desc_create(adamw_desc_t* out, int64_t count, const int64_t* sizes,
                                           conv2d_dtype grad_dtype, adamw_states states, conv2d_dtype copy_dtype) {
    if (!out) return CONV2D_ERR_NULL_PTR;
    *out = nullptr;
    if (count < 0 || count > (1LL << 24) || !known(grad_dtype) || !known(copy_dtype)) return CONV2D_ERR_BAD_PARAM;
    if (states != ADAMW_STATES_F32 && states != ADAMW_STATES_8BIT) return CONV2D_ERR_BAD_PARAM;
    if (count && !sizes) return CONV2D_ERR_NULL_PTR;
    adamw_desc d{};
    d.count = count;
    d.grad = grad_dtype; d.copy = copy_dtype; d.states = states;
    d.beta1 = 0.9; d.beta2 = 0.999; d.eps = 1e-8;
    for (int64_t i = 0; i < count; ++i) {
        // (The kernel numbers blocks of 256 with 32 bits, and an element's group of four.)
        if (sizes[i] < 0 || sizes[i] > (1LL << 34)) return CONV2D_ERR_BAD_PARAM;
        d.elements += (sizes[i] + 255) / 256 * 256;
        if (d.elements >= (1LL << 40)) return CONV2D_ERR_BAD_PARAM;
    }
    d.tensors = new (std::nothrow) adamw_desc::Tensor[count > 0 ? count : 1];
    if (!d.tensors) return CONV2D_ERR_BAD_PARAM;
    int64_t at = 0;
    for (int64_t i = 0; i < count; ++i) {
        d.tensors[i] = adamw_desc::Tensor{sizes[i], at, 0.f};
        at += (sizes[i] + 255) / 256 * 256;
    }
    const conv2d_status s = give(out, d);
    if (s != CONV2D_OK) delete[] d.tensors;
    return s;
}

CONV2D_API conv2d_status adamw_desc_set_rates(adamw_desc_t d, double beta1, double beta2, double eps) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    // As the kernel holds them: 1 - b above zero, eps a normal number.
    if (!(beta1 >= 0.0 && (float)beta1 < 1.f) || !(beta2 >= 0.0 && (float)beta2 < 1.f)) return CONV2D_ERR_BAD_PARAM;
    if (!((float)eps >= 0x1p-126f) || !isfinite((float)eps)) return CONV2D_ERR_BAD_PARAM;
    d->beta1 = beta1;
    d->beta2 = beta2;
    d->eps = eps;
    return CONV2D_OK;
}

CONV2D_API conv2d_status adamw_desc_set_weight_decay(adamw_desc_t d, const float* decay) {
    if (!d) return CONV2D_ERR_NULL_PTR;
    if (d->count && !decay) return CONV2D_ERR_NULL_PTR;
    for (int64_t i = 0; i < d->count; ++i)
        if (!isfinite(decay[i])) return CONV2D_ERR_BAD_PARAM;
    for (int64_t i = 0; i < d->count; ++i) d->tensors[i].decay = decay[i];
    return CONV2D_OK;
}

CONV2D_API conv2d_status adamw_desc_destroy(adamw_desc_t d) {
    if (d) delete[] d->tensors;
    delete d;
    return CONV2D_OK;
}

CONV2D_API conv2d_status adamw_state_elements(adamw_desc_t d, int64_t* elements) {
    if (!d || !elements) return CONV2D_ERR_NULL_PTR;
    *elements = d->elements;
    return CONV2D_OK;
}

CONV2D_API conv2d_status adamw_state_offset(adamw_desc_t d, int64_t i, int64_t* offset) {
    if (!d || !offset) return CONV2D_ERR_NULL_PTR;
    if (i < 0 || i >= d->count) return CONV2D_ERR_BAD_PARAM;
    *offset = d->tensors[i].offset;
    return CONV2D_OK;
}

CONV2D_API conv2d_status adamw_step(adamw_desc_t dp, float* const* params, const void* const* grads,
                                    void* const* copies, void* m, void* v, void* m_scale, void* v_scale, int64_t step,
                                    float lr, const int64_t* device_step, const float* device_lr,
                                    const float* grad_scale, const float* skip, uint64_t seed, void* stream) {
    if (!dp) return CONV2D_ERR_NULL_PTR;
    const adamw_desc& d = *dp;
    if ((!device_step && step < 1) || (!device_lr && !isfinite(lr))) return CONV2D_ERR_BAD_PARAM;
    if (!aligned_to(device_step, 8) || !aligned_to(device_lr, 4) || !aligned_to(grad_scale, 4) || !aligned_to(skip, 4))
        return CONV2D_ERR_MISALIGNED;
    if (d.elements == 0) return CONV2D_OK;
    const bool eight = d.states == ADAMW_STATES_8BIT, copied = d.copy != CONV2D_F32;
    if (!params || !grads || (copied && !copies) || !m || !v || (eight && (!m_scale || !v_scale)))
        return CONV2D_ERR_NULL_PTR;
    if (!aligned_to(m, 32) || !aligned_to(v, 32)) return CONV2D_ERR_MISALIGNED;
    const size_t ge = elem_bytes(d.grad);
    for (int64_t i = 0; i < d.count; ++i) {
        if (!d.tensors[i].n) continue;
        if (!params[i] || !grads[i] || (copied && !copies[i])) return CONV2D_ERR_NULL_PTR;
        if (!aligned_to(params[i], 4) || !aligned_to(grads[i], ge) || (copied && !aligned_to(copies[i], 2)))
            return CONV2D_ERR_MISALIGNED;
    }
    return of(launch_adamw(d, params, grads, copied ? copies : nullptr, m, v, m_scale, v_scale, step, lr, device_step,
                           device_lr, grad_scale, skip, seed, static_cast<cudaStream_t>(stream)));
}
