/*
 * head.h — C ABI of the training-head operators of the GB300 (sm_103a)
 * convolution library: layer norm, dropout, a gated feed-forward block and
 * linear cross entropy, forward and backward, and AdamW.  They take a convolution's output (include/conv2d.h)
 * from feature planes to a loss over a vocabulary, its gradients and the next
 * weights.
 *
 * Conventions are those of conv2d.h: every function returns a conv2d_status
 * and lets no C++ exception out; device pointers belong to the caller; nothing
 * is allocated or retained; `stream` is a cudaStream_t cast to void*, on which
 * all work is queued; descriptors are host memory, can be made without a GPU,
 * and are safe to use from several threads once set up (workspace sizes and
 * launch plans are those of the device that is current when one is made).  Element types are
 * conv2d_dtype; 16-bit values are widened on load, every sum, mean, norm and
 * softmax is held in fp32, and a result is rounded to nearest even once.
 * Waits are bounded as conv2d_set_wait_limit says; layer norm's row kernels look
 * for a copy once, for up to a time slice of the hardware, before the limit
 * counts.
 * Results do not depend on the order in which blocks run: no kernel here
 * accumulates through floating-point atomics, so a call repeated on the same
 * inputs gives the same bits.
 */
#ifndef HEAD_GB300_H
#define HEAD_GB300_H

#include "conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct layernorm_desc *layernorm_desc_t;
typedef struct dropout_desc *dropout_desc_t;
typedef struct linear_ce_desc *linear_ce_desc_t;
typedef struct gated_ffn_desc *gated_ffn_desc_t;
typedef struct adamw_desc *adamw_desc_t;

/* ---------------------------------------------------------------- layer norm
 * Over each of `rows` rows of `cols` elements:
 *   mean = sum x / cols,  rstd = (sum (x - mean)^2 / cols + eps)^(-1/2),
 *   y = (x - mean) rstd gamma + beta.
 * Backward, with z = (x - mean) rstd and a = dy gamma:
 *   dx = rstd (a - sum a / cols - z sum(a z) / cols),
 *   dgamma = sum over rows of dy z,  dbeta = sum over rows of dy. */

/* Create a descriptor.
 *   rows >= 0, cols >= 1; rows and cols at most 2^31-1
 *   dtype        of x, y, dy, dx
 *   param_dtype  of gamma, beta, dgamma, dbeta: dtype or CONV2D_F32
 *   eps >= 0
 * Errors: NULL_PTR, BAD_PARAM. */
conv2d_status layernorm_desc_create(layernorm_desc_t *out, int64_t rows, int64_t cols, conv2d_dtype dtype,
                                    conv2d_dtype param_dtype, float eps);

/* Elements from one row to the next: x_stride of x and dx, y_stride of y and
 * dy (default cols, at least cols; the elements of a row are adjacent).
 * Errors: NULL_PTR, BAD_PARAM; UNSUPPORTED after layernorm_desc_set_planes
 * for an x_stride other than cols. */
conv2d_status layernorm_desc_set_row_strides(layernorm_desc_t d, int64_t x_stride, int64_t y_stride);

/* Read x (and write dx) channels-first, as conv2d_fwd writes its output:
 * [rows / pixels][cols][pixels], normalised over the cols channels of each
 * pixel.  Row i of y, dy, mean and rstd is pixel i % pixels of image
 * i / pixels.  pixels = 0 restores rows.  Errors: NULL_PTR; BAD_PARAM when
 * pixels < 0 or does not divide rows; UNSUPPORTED with an x_stride, and for
 * more than 16384 channels. */
conv2d_status layernorm_desc_set_planes(layernorm_desc_t d, int64_t pixels);

conv2d_status layernorm_desc_destroy(layernorm_desc_t d);

/* Workspace bytes of layernorm_bwd (layernorm_fwd needs none). */
conv2d_status layernorm_workspace_size(layernorm_desc_t d, size_t *bytes);

/* y = layer norm of x.  gamma and beta (cols elements each) may be NULL: 1
 * and 0.  mean and rstd (rows floats each) are written for the backward pass
 * unless NULL.  Pointers need only their element's alignment; 16-byte aligned
 * rows run fastest.  y may be x when their strides agree and x is in rows.
 * Errors: NULL_PTR, MISALIGNED, CUDA. */
conv2d_status layernorm_fwd(layernorm_desc_t d, const void *x, const void *gamma, const void *beta, void *y,
                            float *mean, float *rstd, void *stream);

/* Gradients from dy and the forward pass's x, mean and rstd.  dx, dgamma and
 * dbeta may each be NULL (not wanted).  The workspace (16-byte aligned) is
 * garbage on entry and exit.
 * Errors: NULL_PTR, MISALIGNED, WORKSPACE_TOO_SMALL, CUDA. */
conv2d_status layernorm_bwd(layernorm_desc_t d, const void *dy, const void *x, const void *gamma, const float *mean,
                            const float *rstd, void *dx, void *dgamma, void *dbeta, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------- dropout
 * y = residual + keep x / (1 - p), dx = keep dy / (1 - p).  The mask is never
 * stored: keep of element i (row-major index row * cols + col, whatever the
 * strides) is a function of (seed, offset, i).  With Philox4x32-10 ("Parallel
 * random numbers: as easy as 1, 2, 3", Salmon et al., 2011) under key = seed
 * (low word first) and counter = (b mod 2^32, b div 2^32, offset mod 2^32,
 * offset div 2^32 + 2^31 s), b = i div 8, the four output words read as eight
 * 16-bit words (low half first) give, at word i mod 8, the high half (s = 0)
 * and the low half (s = 1) of a uniform 32-bit number; the element is dropped
 * where it is below round(p 2^32).  Calls that should draw different masks
 * take different offsets. */

/* Create a descriptor.  rows >= 0, cols >= 1, 0 <= p <= 1 (p = 1 drops all).
 * Errors: NULL_PTR, BAD_PARAM. */
conv2d_status dropout_desc_create(dropout_desc_t *out, int64_t rows, int64_t cols, conv2d_dtype dtype, double p);

/* Elements from one row to the next: x_stride of x and dx, residual_stride,
 * y_stride of y and dy (defaults cols, each at least cols). */
conv2d_status dropout_desc_set_row_strides(dropout_desc_t d, int64_t x_stride, int64_t residual_stride,
                                           int64_t y_stride);

conv2d_status dropout_desc_destroy(dropout_desc_t d);

/* y from x and residual (NULL: none).  y may be x or residual when their
 * strides agree.  offset < 2^63.  Errors: NULL_PTR, BAD_PARAM, MISALIGNED
 * (element alignment), CUDA. */
conv2d_status dropout_fwd(dropout_desc_t d, const void *x, const void *residual, void *y, uint64_t seed,
                          uint64_t offset, void *stream);

/* dx from dy with the mask of dropout_fwd under the same seed and offset (the
 * residual's gradient is dy itself).  Errors as dropout_fwd. */
conv2d_status dropout_bwd(dropout_desc_t d, const void *dy, void *dx, uint64_t seed, uint64_t offset, void *stream);

/* ------------------------------------------------------- linear cross entropy
 * For each of `tokens` rows h_n of h and its target y_n, over the `vocab` rows
 * w_v of w:
 *   z_nv = h_n . w_v,  lse_n = log sum_v exp z_nv,  loss_n = lse_n - z_{n,y_n},
 * and loss_n = 0 where y_n is the ignored index.  The logits z are never kept:
 * the forward pass reduces each tile of them where it is computed, the
 * backward pass recomputes them in pieces of the vocabulary.
 *   dz_nv = g_n (exp(z_nv - lse_n) - [v = y_n]),  dh = dz w,  dw = dz^T h,
 * with g_n = 0 for ignored targets.  fp16 and bf16 run on the tensor cores
 * with fp32 accumulation, and dz is rounded to that type for the two products
 * of the backward pass (to two parts of that type, twice its bits, up to 256
 * tokens).  The tensor cores truncate their fp32 sums: over the 16384 (fp16) or
 * 131072 (bf16) terms that are summed there at most before the sums go on
 * rounded to nearest, terms of one sign lose up to a fifth of the result type's
 * unit roundoff.  fp32 runs on the tensor cores too: each value is the
 * sum of three bf16 parts (8 bits of the significand each), and the six
 * leading products of the parts, exact in fp32, are accumulated; an infinity
 * in h or w makes its logits NaN there (a part of the other factor is zero). */

typedef enum { HEAD_REDUCE_NONE = 0, HEAD_REDUCE_SUM = 1, HEAD_REDUCE_MEAN = 2 } head_reduction;

/* Create a descriptor.
 *   0 <= tokens <= 2^30, 1 <= hidden <= 2^26, 1 <= vocab <= 2^30, and fewer
 *                 than 2^31 tiles of 128 tokens by 64 vocabulary rows
 *   reduction     NONE: loss and dloss have `tokens` values; SUM and MEAN
 *                 (over the targets that are not ignored; 0 when all are): one
 *   ignore_index  target value whose rows neither cost nor train
 * Errors: NULL_PTR, BAD_PARAM. */
conv2d_status linear_ce_desc_create(linear_ce_desc_t *out, int64_t tokens, int64_t hidden, int64_t vocab,
                                    conv2d_dtype dtype, head_reduction reduction, int64_t ignore_index);

/* Elements from one row to the next of h and w (defaults hidden, at least
 * hidden; dh and dw are always contiguous).  h or w whose row stride is no
 * multiple of 8 elements, or fp32, is first copied into the workspace in the
 * layout the tensor cores read.  Changes the workspace sizes. */
conv2d_status linear_ce_desc_set_row_strides(linear_ce_desc_t d, int64_t h_stride, int64_t w_stride);

/* Vocabulary rows per piece of the backward pass (rounded up to a multiple of
 * 256; 0 = automatic: the widest piece whose dz stays within 256 MiB).
 * Smaller pieces need less workspace.  Changes the workspace size. */
conv2d_status linear_ce_desc_set_piece(linear_ce_desc_t d, int64_t vocab_rows);

/* 16-bit parts in which dz of fp16 and bf16 operands is kept: 1, or 2 for twice
 * its bits, which leaves dh and dw with little more than their own rounding (dz
 * takes twice the memory, and the two products of the backward pass twice the
 * time; with one part the rounding of dz adds up to as much again as theirs,
 * where a row's sum is mostly one term).  0 = automatic: 2 up to 256 tokens, where the rounding of dz does not
 * average out, else 1.  Changes the workspace size.  Errors: NULL_PTR;
 * BAD_PARAM; UNSUPPORTED for fp32 (always three parts) unless 0. */
conv2d_status linear_ce_desc_set_dz_parts(linear_ce_desc_t d, int parts);

conv2d_status linear_ce_desc_destroy(linear_ce_desc_t d);

/* Workspace bytes of linear_ce_fwd and of linear_ce_bwd (either may be NULL). */
conv2d_status linear_ce_workspace_size(linear_ce_desc_t d, size_t *fwd_bytes, size_t *bwd_bytes);

/* Losses and log-sum-exps.
 *   h [tokens][hidden], w [vocab][hidden], target [tokens] int64
 *   loss  tokens floats or one (see reduction);  lse  tokens floats
 * A target that is neither in [0, vocab) nor the ignored index makes its
 * row's loss NaN (and with it the sum or mean) and counts as ignored in the
 * mean and in linear_ce_bwd.
 * h and w (read in place unless the row stride or type forces a copy) and the
 * workspace are 16-byte aligned.  Errors: NULL_PTR, MISALIGNED,
 * WORKSPACE_TOO_SMALL, CUDA; bounded waits that expire are reported by
 * conv2d_device_status. */
conv2d_status linear_ce_fwd(linear_ce_desc_t d, const void *h, const void *w, const int64_t *target, float *loss,
                            float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* dh [tokens][hidden] and dw [vocab][hidden], of the descriptor's type, from
 * the forward pass's lse and dloss (tokens floats, or one).  Either of dh and
 * dw may be NULL (not wanted).  Errors as linear_ce_fwd. */
conv2d_status linear_ce_bwd(linear_ce_desc_t d, const void *h, const void *w, const int64_t *target, const float *lse,
                            const float *dloss, void *dh, void *dw, void *workspace, size_t workspace_bytes,
                            void *stream);

/* ------------------------------------------------- gated feed-forward block
 * For each of `tokens` rows of x (`hidden` columns), with Wg and Wu
 * [inner][hidden] and Wd [hidden][inner]:
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = residual + h Wd^T,
 * act(g) = g / (1 + exp(-g)) (SILU), g Phi(g) (GELU, Phi the normal
 * distribution) or g / (1 + exp(-2 sqrt(2/pi) (g + 0.044715 g^3))) (GELU_TANH).
 * Backward, from dy and the saved g, u and h:
 *   dh = dy Wd,  dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu,
 *   dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h    (the residual's gradient is dy).
 * fp16 and bf16 run on the tensor cores with fp32 accumulation; g, u and dh stay
 * in fp32, while h, dg and du are rounded to the operands' type for the products
 * that read them (fp16: dg and du held times a power of two that takes the largest
 * finite one to [2^10, 2^15), whatever dy's size: only those below 2^-24 of it may lose
 * digits; an h beyond fp16's range is infinite).  fp32 runs there
 * too, as three bf16 parts a value and the six leading products of the parts; an
 * infinity in an operand makes what it enters NaN.  Forward passes of few tokens run
 * on the CUDA cores and keep h in fp32. */

typedef enum { FFN_SILU = 0, FFN_GELU = 1, FFN_GELU_TANH = 2 } gated_ffn_act;

/* Create a descriptor.
 *   0 <= tokens <= 2^30, 1 <= hidden <= 16384, 1 <= inner <= 2^20, and fewer than
 *   2^31 tiles of 128 tokens by 32 inner columns
 * Errors: NULL_PTR, BAD_PARAM. */
conv2d_status gated_ffn_desc_create(gated_ffn_desc_t *out, int64_t tokens, int64_t hidden, int64_t inner,
                                    conv2d_dtype dtype, gated_ffn_act act);

/* Elements from one row to the next of x, and of y, residual and dy (defaults
 * hidden, at least hidden; dx, the weights and their gradients are contiguous).
 * Operands whose rows are no multiple of 8 elements apart, and fp32 ones, are first
 * copied into the workspace in the layout the tensor cores read.  Changes the
 * workspace sizes. */
conv2d_status gated_ffn_desc_set_row_strides(gated_ffn_desc_t d, int64_t x_stride, int64_t y_stride);

conv2d_status gated_ffn_desc_destroy(gated_ffn_desc_t d);

/* Workspace bytes of gated_ffn_fwd and gated_ffn_bwd, and bytes of `saved` (each may be NULL). */
conv2d_status gated_ffn_workspace_size(gated_ffn_desc_t d, size_t *fwd_bytes, size_t *bwd_bytes, size_t *saved_bytes);

/* y from x, the weights and residual (NULL: none).  y may be residual, and x where
 * their strides agree.  saved (NULL: not wanted) receives g and u (fp32) and h for the
 * backward pass, in an order of its own, 32-byte aligned.  x and the weights
 * are 16-byte aligned (those that are copied, and all of fp32: as their elements), the workspace too.
 * Errors: NULL_PTR, MISALIGNED, WORKSPACE_TOO_SMALL, CUDA; UNSUPPORTED for more
 * tiles and splits than 2^31; bounded waits that expire are reported by
 * conv2d_device_status. */
conv2d_status gated_ffn_fwd(gated_ffn_desc_t d, const void *x, const void *wg, const void *wu, const void *wd,
                            const void *residual, void *y, float *saved, void *workspace, size_t workspace_bytes,
                            void *stream);

/* Gradients from dy and what gated_ffn_fwd saved for the same x and weights.  Each of dx
 * [tokens][hidden], dwg, dwu and dwd may be NULL (not wanted); none overlaps an operand.
 * Errors as gated_ffn_fwd. */
conv2d_status gated_ffn_bwd(gated_ffn_desc_t d, const void *dy, const void *x, const void *wg, const void *wu,
                            const void *wd, const float *saved, void *dx, void *dwg, void *dwu, void *dwd,
                            void *workspace, size_t workspace_bytes, void *stream);

/* --------------------------------------------------------------------- AdamW
 * A step of `count` tensors at once, in place.  With g the gradient times
 * *grad_scale, for each element:
 *   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
 *   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
 * t the step's number, from 1 on; the copy (fp16 or bf16) is p rounded.  The
 * parameters are fp32.  The moments of all tensors lie one tensor after the
 * other in one buffer each, every tensor's in whole blocks of 256
 * (adamw_state_offset); zero in all their bytes before the first step.
 * In 8 bits a block's values are its codes (m e4m3, v e5m2, as of the OCP 8-bit
 * formats) times its scale 2^(byte - 127): the scale takes the largest value to
 * the type's top binade, at most 1.75 there, and each value goes to one of its
 * neighbours, up where the bits that are left over and 16 random bits of the
 * same weight make a carry; v above zero is never stored as zero.  The random
 * bits of element i of tensor k in step t are the halves (low: m, high: v) of
 * word i mod 4 of Philox4x32-10 under key = seed and counter = (i div 4, k,
 * t mod 2^32, t div 2^32).  p takes the moments before they are rounded.  A block
 * with an infinity or a NaN gets the scale 255: all its values are NaN from
 * the next step on. */

typedef enum { ADAMW_STATES_F32 = 0, ADAMW_STATES_8BIT = 1 } adamw_states;

/* Create a descriptor of `count` tensors of sizes[i] elements.
 *   0 <= count <= 2^24, 0 <= sizes[i] <= 2^34, fewer than 2^40 together
 *   grad_dtype   of all gradients
 *   copy_dtype   of all copies: CONV2D_F16 or CONV2D_BF16; CONV2D_F32: no copies
 * b1 = 0.9, b2 = 0.999, eps = 1e-8 and no decay until set.
 * Errors: NULL_PTR, BAD_PARAM. */
conv2d_status adamw_desc_create(adamw_desc_t *out, int64_t count, const int64_t *sizes, conv2d_dtype grad_dtype,
                                adamw_states states, conv2d_dtype copy_dtype);

/* 0 <= beta1, beta2 < 1 and eps >= 2^-126 (as fp32).  Errors: NULL_PTR, BAD_PARAM. */
conv2d_status adamw_desc_set_rates(adamw_desc_t d, double beta1, double beta2, double eps);

/* The decay of each tensor (count values, finite).  Errors: NULL_PTR, BAD_PARAM. */
conv2d_status adamw_desc_set_weight_decay(adamw_desc_t d, const float *decay);

conv2d_status adamw_desc_destroy(adamw_desc_t d);

/* Elements of each moment's buffer (a multiple of 256; the scales are one byte
 * for each 256), and the first one of tensor i. */
conv2d_status adamw_state_elements(adamw_desc_t d, int64_t *elements);
conv2d_status adamw_state_offset(adamw_desc_t d, int64_t i, int64_t *offset);

/* One step.
 *   params, grads, copies   host arrays of `count` device addresses (read before
 *                the call returns; those of empty tensors are ignored); copies is
 *                NULL where the descriptor has none.  Elements are adjacent and
 *                need only their own alignment (32-byte aligned ones, 16 of
 *                16-bit types, run fastest).  No two tensors overlap.
 *   m, v         the moments, 32-byte aligned; m_scale, v_scale theirs in 8 bits (else ignored)
 *   step, lr     t >= 1 and a finite rate, unless the device holds them:
 *   device_step, device_lr   NULL, or addresses that the step reads instead, so
 *                that a captured call goes on where the program sets them
 *   grad_scale   NULL, or the address of the factor of all gradients
 *   skip         NULL, or the address of a float: unless it is 0, nothing changes
 * Errors: NULL_PTR, BAD_PARAM, MISALIGNED, CUDA. */
conv2d_status adamw_step(adamw_desc_t d, float *const *params, const void *const *grads, void *const *copies, void *m,
                         void *v, void *m_scale, void *v_scale, int64_t step, float lr, const int64_t *device_step,
                         const float *device_lr, const float *grad_scale, const float *skip, uint64_t seed,
                         void *stream);

#ifdef __cplusplus
}
#endif
#endif /* HEAD_GB300_H */
