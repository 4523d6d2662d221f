"""PyTorch-tensor convenience layer over the training-head operators.

Layer norm, dropout and linear cross entropy take a convolution's features to
a loss over a vocabulary and its gradients.  As in ``conv``, PyTorch provides
device memory and the current stream, every arithmetic step runs in the
library's kernels, and shapes are checked so that a wrong tensor fails with a
Python error instead of a bad pointer.  Each class is one problem shape:
calling it runs the forward pass, ``backward`` the gradients.
"""
from __future__ import annotations

import functools

import torch

from . import head_capi
from .conv import _NAME, _TORCH_DTYPE


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _on_stream(f):
    """Accept stream=: the call and the tensors that it allocates belong to that stream."""
    @functools.wraps(f)
    def call(self, *args, stream=None, **kwargs):
        if stream is None:
            return f(self, *args, **kwargs)
        with torch.cuda.stream(stream):
            return f(self, *args, **kwargs)
    return call


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _check_rows(name, t, rows, cols, stride, dtype):
    """A (rows, cols) tensor whose rows are `stride` elements apart."""
    if (t.dtype != _TORCH_DTYPE[dtype] or t.shape != (rows, cols)
            or not (t.stride() == (stride, 1) or _same_rows(t, rows, cols, stride))):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(rows, cols)} with rows {stride} elements apart")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _same_rows(t, rows, cols, stride):
    # Strides of dimensions of size one (or of empty tensors) mean nothing.
    return (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) == stride)


def _check_flat(name, t, shape, dtype):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype} and shape {tuple(shape)}")


class _Op:
    """A descriptor, destroyed with its owner."""
    _destroy = None

    def __del__(self):
        d = getattr(self, "desc", None)
        if d:
            try:
                type(self)._destroy(d)
            except Exception:
                pass
            self.desc = None


class LayerNorm(_Op):
    """Layer norm of (rows, cols), or of channels-first planes.

    pixels     x (and dx) are planes [rows / pixels][cols][pixels], the layout
               conv2d writes, normalised over channels; y and dy are rows
    x_stride, y_stride   elements between rows of x and dx, y and dy
    """
    _destroy = staticmethod(head_capi.layernorm_desc_destroy)

    def __init__(self, rows, cols, dtype="f32", param_dtype=None, eps=1e-5, pixels=None, x_stride=None, y_stride=None):
        self.rows, self.cols, self.dtype = rows, cols, dtype
        self.param_dtype = param_dtype or dtype
        self.pixels = pixels
        self.x_stride, self.y_stride = x_stride or cols, y_stride or cols
        self.desc = head_capi.layernorm_desc_create(rows, cols, dtype, self.param_dtype, eps)
        if self.x_stride != cols or self.y_stride != cols:
            head_capi.layernorm_desc_set_row_strides(self.desc, self.x_stride, self.y_stride)
        if pixels:
            head_capi.layernorm_desc_set_planes(self.desc, pixels)
        self.workspace_bytes = head_capi.layernorm_workspace_size(self.desc)

    def _check_x(self, name, x):
        if not self.pixels:
            _check_rows(name, x, self.rows, self.cols, self.x_stride, self.dtype)
            return
        want = (self.rows // self.pixels, self.cols)
        if (x.dim() < 3 or tuple(x.shape[:2]) != want or x[0, 0].numel() != self.pixels if x.numel() else False) \
                or x.numel() != self.rows * self.cols or x.dtype != _TORCH_DTYPE[self.dtype] \
                or not x.is_contiguous() or not x.is_cuda:
            raise ValueError(f"{name} must be contiguous {self.dtype} planes of shape {want} + pixels, "
                             f"{self.pixels} pixels each")

    def _check_params(self, *named):
        for name, t in named:
            if t is not None:
                _check_flat(name, t, (self.cols,), _TORCH_DTYPE[self.param_dtype])

    def _like_x(self, x):
        if self.pixels:
            return torch.empty_like(x)
        return torch.empty_strided((self.rows, self.cols), (self.x_stride, 1), dtype=x.dtype, device=x.device)

    @_on_stream
    def __call__(self, x, gamma=None, beta=None, y=None, stats=False):
        """y, or (y, mean, rstd) with `stats` (what `backward` needs)."""
        self._check_x("x", x)
        self._check_params(("gamma", gamma), ("beta", beta))
        if y is None:
            y = torch.empty_strided((self.rows, self.cols), (self.y_stride, 1), dtype=x.dtype, device=x.device)
        else:
            _check_rows("y", y, self.rows, self.cols, self.y_stride, self.dtype)
        mean = rstd = None
        if stats:
            mean, rstd = torch.empty((2, self.rows), dtype=torch.float32, device=x.device).unbind(0)
        head_capi.layernorm_fwd(self.desc, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                                _stream(x.device))
        return (y, mean, rstd) if stats else y

    @_on_stream
    def backward(self, dy, x, gamma, mean, rstd, need_dx=True, need_params=True, workspace=None):
        """(dx, dgamma, dbeta); None in the place of what is not needed."""
        self._check_x("x", x)
        _check_rows("dy", dy, self.rows, self.cols, self.y_stride, self.dtype)
        self._check_params(("gamma", gamma))
        _check_flat("mean", mean, (self.rows,), torch.float32)
        _check_flat("rstd", rstd, (self.rows,), torch.float32)
        dx = self._like_x(x) if need_dx else None
        dgamma = dbeta = None
        if need_params:
            dgamma, dbeta = torch.empty((2, self.cols), dtype=_TORCH_DTYPE[self.param_dtype],
                                        device=x.device).unbind(0)
        if workspace is None:
            workspace = torch.empty(max(self.workspace_bytes, 1), dtype=torch.uint8, device=x.device)
        head_capi.layernorm_bwd(self.desc, _ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                                _ptr(dgamma), _ptr(dbeta), _ptr(workspace), workspace.numel(),
                                _stream(x.device))
        return dx, dgamma, dbeta


class Dropout(_Op):
    """Dropout of (rows, cols) with probability p.  The mask is a function of
    (seed, offset) and the element's index, so `backward` redraws it."""
    _destroy = staticmethod(head_capi.dropout_desc_destroy)

    def __init__(self, rows, cols, dtype="f32", p=0.5, x_stride=None, residual_stride=None, y_stride=None):
        self.rows, self.cols, self.dtype, self.p = rows, cols, dtype, p
        self.x_stride, self.residual_stride, self.y_stride = x_stride or cols, residual_stride or cols, y_stride or cols
        self.desc = head_capi.dropout_desc_create(rows, cols, dtype, p)
        if (self.x_stride, self.residual_stride, self.y_stride) != (cols, cols, cols):
            head_capi.dropout_desc_set_row_strides(self.desc, self.x_stride, self.residual_stride, self.y_stride)

    @_on_stream
    def __call__(self, x, seed, offset=0, residual=None, y=None):
        """residual + dropped x (y may be x or residual)."""
        _check_rows("x", x, self.rows, self.cols, self.x_stride, self.dtype)
        if residual is not None:
            _check_rows("residual", residual, self.rows, self.cols, self.residual_stride, self.dtype)
        if y is None:
            y = torch.empty_strided((self.rows, self.cols), (self.y_stride, 1), dtype=x.dtype, device=x.device)
        else:
            _check_rows("y", y, self.rows, self.cols, self.y_stride, self.dtype)
        head_capi.dropout_fwd(self.desc, _ptr(x), _ptr(residual), _ptr(y), seed, offset, _stream(x.device))
        return y

    @_on_stream
    def backward(self, dy, seed, offset=0, dx=None):
        """dx under the mask of the forward call with the same seed and offset."""
        _check_rows("dy", dy, self.rows, self.cols, self.y_stride, self.dtype)
        if dx is None:
            dx = torch.empty_strided((self.rows, self.cols), (self.x_stride, 1), dtype=dy.dtype, device=dy.device)
        else:
            _check_rows("dx", dx, self.rows, self.cols, self.x_stride, self.dtype)
        head_capi.dropout_bwd(self.desc, _ptr(dy), _ptr(dx), seed, offset, _stream(dy.device))
        return dx


class LinearCrossEntropy(_Op):
    """Softmax cross entropy of h w^T against targets, without keeping the logits.

    h (tokens, hidden), w (vocab, hidden), target (tokens,) int64
    reduction  "none", "sum" or "mean" (over targets other than ignore_index)
    piece      vocabulary rows per step of the backward pass (None: automatic)
    """
    _destroy = staticmethod(head_capi.linear_ce_desc_destroy)

    def __init__(self, tokens, hidden, vocab, dtype="bf16", reduction="mean", ignore_index=-100, h_stride=None,
                 w_stride=None, piece=None):
        self.tokens, self.hidden, self.vocab, self.dtype, self.reduction = tokens, hidden, vocab, dtype, reduction
        self.h_stride, self.w_stride = h_stride or hidden, w_stride or hidden
        self.desc = head_capi.linear_ce_desc_create(tokens, hidden, vocab, dtype, reduction, ignore_index)
        if self.h_stride != hidden or self.w_stride != hidden:
            head_capi.linear_ce_desc_set_row_strides(self.desc, self.h_stride, self.w_stride)
        if piece:
            head_capi.linear_ce_desc_set_piece(self.desc, piece)
        self.workspace_bytes, self.backward_workspace_bytes = head_capi.linear_ce_workspace_size(self.desc)

    @property
    def loss_shape(self):
        return (self.tokens,) if self.reduction == "none" else ()

    def _check(self, h, w, target):
        _check_rows("h", h, self.tokens, self.hidden, self.h_stride, self.dtype)
        _check_rows("w", w, self.vocab, self.hidden, self.w_stride, self.dtype)
        _check_flat("target", target, (self.tokens,), torch.int64)

    @_on_stream
    def __call__(self, h, w, target, workspace=None):
        """(loss, lse): lse (log-sum-exp per token) is what `backward` needs."""
        self._check(h, w, target)
        loss = torch.empty(self.loss_shape, dtype=torch.float32, device=h.device)
        lse = torch.empty((self.tokens,), dtype=torch.float32, device=h.device)
        if workspace is None:
            workspace = torch.empty(max(self.workspace_bytes, 1), dtype=torch.uint8, device=h.device)
        head_capi.linear_ce_fwd(self.desc, _ptr(h), _ptr(w), _ptr(target), _ptr(loss), _ptr(lse), _ptr(workspace),
                                workspace.numel(), _stream(h.device))
        return loss, lse

    @_on_stream
    def backward(self, h, w, target, lse, dloss, need_dh=True, need_dw=True, workspace=None):
        """(dh, dw); None in the place of what is not needed."""
        self._check(h, w, target)
        _check_flat("lse", lse, (self.tokens,), torch.float32)
        _check_flat("dloss", dloss, self.loss_shape, torch.float32)
        dh = torch.empty((self.tokens, self.hidden), dtype=h.dtype, device=h.device) if need_dh else None
        dw = torch.empty((self.vocab, self.hidden), dtype=w.dtype, device=w.device) if need_dw else None
        if workspace is None:
            workspace = torch.empty(max(self.backward_workspace_bytes, 1), dtype=torch.uint8, device=h.device)
        head_capi.linear_ce_bwd(self.desc, _ptr(h), _ptr(w), _ptr(target), _ptr(lse), _ptr(dloss), _ptr(dh), _ptr(dw),
                                _ptr(workspace), workspace.numel(), _stream(h.device))
        return dh, dw


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """y of a contiguous (rows, cols) tensor on the current stream."""
    param = _NAME[gamma.dtype] if gamma is not None else _NAME[beta.dtype] if beta is not None else None
    return LayerNorm(x.shape[0], x.shape[1], _NAME[x.dtype], param, eps)(x, gamma, beta)


def dropout(x, p, seed, offset=0, residual=None):
    """residual + dropped x of a contiguous (rows, cols) tensor on the current stream."""
    return Dropout(x.shape[0], x.shape[1], _NAME[x.dtype], p)(x, seed, offset, residual)


def linear_cross_entropy(h, w, target, reduction="mean", ignore_index=-100):
    """The loss of contiguous h and w on the current stream."""
    op = LinearCrossEntropy(h.shape[0], h.shape[1], w.shape[0], _NAME[h.dtype], reduction, ignore_index)
    return op(h, w, target)[0]
