"""PyTorch-tensor convenience layer over the training-head operators.

Layer norm, dropout and linear cross entropy take a convolution's features to
a loss over a vocabulary and its gradients.  As in ``conv``, PyTorch provides
device memory and the current stream, every arithmetic step runs in the
library's kernels, and shapes and devices are checked so that a wrong tensor
fails with a Python error instead of a bad pointer.  Each class is one problem
shape: calling it runs the forward pass, ``backward`` the gradients.  All tensors
of a call, its workspace among them, are on one GPU, on which it runs whichever
is current.  With stream= (of that GPU) a call and the tensors that it allocates
belong to that stream.  No call records an autograd graph: gradients come from
``backward``, and results carry none, whatever requires_grad their inputs have.
"""
from __future__ import annotations

import torch

from . import head_capi
from .conv import _NAME, _TORCH_DTYPE


_raw_stream = torch._C._cuda_getCurrentRawStream      # the current stream's handle by device index
_current_device = torch._C._cuda_getDevice


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _place(dev, stream):
    """The context in which a call on GPU `dev` belongs: its stream, or that GPU."""
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on GPU {stream.device.index}, the tensors are on GPU {dev}")
    return torch.cuda.stream(stream)


def _check_workspace(t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous buffer on GPU {dev}")


class _Rows:
    """The (rows, cols) tensors of one type whose rows are `stride` elements apart."""

    def __init__(self, rows, cols, stride, dtype):
        self.shape, self.strides, self.name, self.dtype = (rows, cols), (stride, 1), dtype, _TORCH_DTYPE[dtype]

    def check(self, name, t, dev):
        if t.dtype is self.dtype and t.shape == self.shape and t.get_device() == dev:
            s = t.stride()
            if s == self.strides:
                return
            # The stride of a dimension of size one (or of an empty tensor) means nothing.
            if ((self.shape[0] <= 1 or s[0] == self.strides[0]) and (self.shape[1] <= 1 or s[1] == 1)) or t.numel() == 0:
                return
        raise ValueError(f"{name} must be a CUDA {self.name} tensor of shape {self.shape} with rows "
                         f"{self.strides[0]} elements apart, on the device of the others")

    def new(self, device):
        if self.strides[0] == self.shape[1]:
            return torch.empty(self.shape, dtype=self.dtype, device=device)
        return torch.empty_strided(self.shape, self.strides, dtype=self.dtype, device=device)


class _Planes:
    """Contiguous channels-first planes: (images, cols, *pixels)."""

    def __init__(self, rows, cols, pixels, dtype):
        self.lead, self.count, self.name, self.dtype = (rows // pixels, cols), rows * cols, dtype, _TORCH_DTYPE[dtype]
        self.pixels = pixels

    def check(self, name, t, dev):
        if t.dtype is not self.dtype or t.dim() < 3 or t.shape[:2] != self.lead or t.numel() != self.count \
                or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{name} must be contiguous CUDA {self.name} planes of shape {self.lead} and {self.pixels} "
                             f"pixels, on the device of the others")


class _Flat:
    """The contiguous tensors of one shape and type."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype = shape, dtype

    def check(self, name, t, dev):
        if t.dtype is not self.dtype or t.shape != self.shape or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{name} must be a contiguous CUDA tensor of {self.dtype} and shape {self.shape}, on the "
                             f"device of the others")

    def new(self, device):
        return torch.empty(self.shape, dtype=self.dtype, device=device)


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
        self._x = _Planes(rows, cols, pixels, dtype) if pixels else _Rows(rows, cols, self.x_stride, dtype)
        self._y = _Rows(rows, cols, self.y_stride, dtype)
        self._param, self._stat = _Flat((cols,), _TORCH_DTYPE[self.param_dtype]), _Flat((rows,), torch.float32)

    def __call__(self, x, gamma=None, beta=None, y=None, stats=False, stream=None):
        """y, or (y, mean, rstd) with `stats` (what `backward` needs)."""
        dev = x.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self(x, gamma, beta, y, stats)
        self._x.check("x", x, dev)
        g = b = mp = rp = 0
        if gamma is not None:
            self._param.check("gamma", gamma, dev)
            g = gamma.data_ptr()
        if beta is not None:
            self._param.check("beta", beta, dev)
            b = beta.data_ptr()
        if y is None:
            y = self._y.new(x.device)
        else:
            self._y.check("y", y, dev)
        if stats:
            mean, rstd = self._stat.new(x.device), self._stat.new(x.device)
            mp, rp = mean.data_ptr(), rstd.data_ptr()
        head_capi.layernorm_fwd(self.desc, x.data_ptr(), g, b, y.data_ptr(), mp, rp, _raw_stream(dev))
        return (y, mean, rstd) if stats else y

    def backward(self, dy, x, gamma, mean, rstd, need_dx=True, need_params=True, workspace=None, stream=None):
        """(dx, dgamma, dbeta); None in the place of what is not needed."""
        dev = x.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self.backward(dy, x, gamma, mean, rstd, need_dx, need_params, workspace)
        self._x.check("x", x, dev)
        self._y.check("dy", dy, dev)
        self._stat.check("mean", mean, dev)
        self._stat.check("rstd", rstd, dev)
        g = xp = gp = bp = 0
        if gamma is not None:
            self._param.check("gamma", gamma, dev)
            g = gamma.data_ptr()
        at = x.device
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=at)
        else:
            _check_workspace(workspace, dev)
        dx = dgamma = dbeta = None
        if need_dx:
            dx = torch.empty_like(x) if self.pixels else self._x.new(at)
            xp = dx.data_ptr()
        if need_params:
            dgamma, dbeta = self._param.new(at), self._param.new(at)
            gp, bp = dgamma.data_ptr(), dbeta.data_ptr()
        head_capi.layernorm_bwd(self.desc, dy.data_ptr(), x.data_ptr(), g, mean.data_ptr(), rstd.data_ptr(), xp, gp, bp,
                                workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
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
        self._x, self._y = _Rows(rows, cols, self.x_stride, dtype), _Rows(rows, cols, self.y_stride, dtype)
        self._residual = _Rows(rows, cols, self.residual_stride, dtype)

    def __call__(self, x, seed, offset=0, residual=None, y=None, stream=None):
        """residual + dropped x (y may be x or residual)."""
        dev = x.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self(x, seed, offset, residual, y)
        self._x.check("x", x, dev)
        if residual is not None:
            self._residual.check("residual", residual, dev)
        if y is None:
            y = self._y.new(x.device)
        else:
            self._y.check("y", y, dev)
        head_capi.dropout_fwd(self.desc, x.data_ptr(), _ptr(residual), y.data_ptr(), seed, offset,
                              _raw_stream(dev))
        return y

    def backward(self, dy, seed, offset=0, dx=None, stream=None):
        """dx under the mask of the forward call with the same seed and offset."""
        dev = dy.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self.backward(dy, seed, offset, dx)
        self._y.check("dy", dy, dev)
        if dx is None:
            dx = self._x.new(dy.device)
        else:
            self._x.check("dx", dx, dev)
        head_capi.dropout_bwd(self.desc, dy.data_ptr(), dx.data_ptr(), seed, offset, _raw_stream(dev))
        return dx


class LinearCrossEntropy(_Op):
    """Softmax cross entropy of h w^T against targets, without keeping the logits.

    h (tokens, hidden), w (vocab, hidden), target (tokens,) int64
    reduction  "none", "sum" or "mean" (over targets other than ignore_index)
    piece      vocabulary rows per step of the backward pass (None: automatic)
    dz_parts   16-bit parts of the logits' gradient, 1 or 2 (None: automatic; fp32 has three)
    """
    _destroy = staticmethod(head_capi.linear_ce_desc_destroy)

    def __init__(self, tokens, hidden, vocab, dtype="bf16", reduction="mean", ignore_index=-100, h_stride=None,
                 w_stride=None, piece=None, dz_parts=None):
        self.tokens, self.hidden, self.vocab, self.dtype, self.reduction = tokens, hidden, vocab, dtype, reduction
        self.h_stride, self.w_stride = h_stride or hidden, w_stride or hidden
        self.desc = head_capi.linear_ce_desc_create(tokens, hidden, vocab, dtype, reduction, ignore_index)
        if self.h_stride != hidden or self.w_stride != hidden:
            head_capi.linear_ce_desc_set_row_strides(self.desc, self.h_stride, self.w_stride)
        if piece:
            head_capi.linear_ce_desc_set_piece(self.desc, piece)
        if dz_parts:
            head_capi.linear_ce_desc_set_dz_parts(self.desc, dz_parts)
        self.workspace_bytes, self.backward_workspace_bytes = head_capi.linear_ce_workspace_size(self.desc)
        self.loss_shape = (tokens,) if reduction == "none" else ()
        self._h, self._w = _Rows(tokens, hidden, self.h_stride, dtype), _Rows(vocab, hidden, self.w_stride, dtype)
        self._target, self._lse = _Flat((tokens,), torch.int64), _Flat((tokens,), torch.float32)
        self._loss = _Flat(self.loss_shape, torch.float32)

    def _check(self, h, w, target, dev):
        self._h.check("h", h, dev)
        self._w.check("w", w, dev)
        self._target.check("target", target, dev)

    def __call__(self, h, w, target, workspace=None, stream=None):
        """(loss, lse): lse (log-sum-exp per token) is what `backward` needs."""
        dev = h.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self(h, w, target, workspace)
        self._check(h, w, target, dev)
        at = h.device
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=at)
        else:
            _check_workspace(workspace, dev)
        loss, lse = self._loss.new(at), self._lse.new(at)
        head_capi.linear_ce_fwd(self.desc, h.data_ptr(), w.data_ptr(), target.data_ptr(), loss.data_ptr(),
                                lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
        return loss, lse

    def backward(self, h, w, target, lse, dloss, need_dh=True, need_dw=True, workspace=None, stream=None):
        """(dh, dw); None in the place of what is not needed."""
        dev = h.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self.backward(h, w, target, lse, dloss, need_dh, need_dw, workspace)
        self._check(h, w, target, dev)
        self._lse.check("lse", lse, dev)
        self._loss.check("dloss", dloss, dev)
        at = h.device
        if workspace is None:
            workspace = torch.empty(self.backward_workspace_bytes, dtype=torch.uint8, device=at)
        else:
            _check_workspace(workspace, dev)
        dh = torch.empty((self.tokens, self.hidden), dtype=h.dtype, device=at) if need_dh else None
        dw = torch.empty((self.vocab, self.hidden), dtype=w.dtype, device=at) if need_dw else None
        head_capi.linear_ce_bwd(self.desc, h.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(),
                                dloss.data_ptr(), _ptr(dh), _ptr(dw), workspace.data_ptr(), workspace.numel(),
                                _raw_stream(dev))
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
