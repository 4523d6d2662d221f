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

import collections
import operator

import torch

from . import head_capi
from .conv import _NAME, _TORCH_DTYPE


_raw_stream = torch._C._cuda_getCurrentRawStream      # the current stream's handle by device index
_current_device = torch._C._cuda_getDevice
_dtype_of = operator.attrgetter("dtype")


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


class GatedFeedForward(_Op):
    """A gated feed-forward block: y = residual + (act(x wg') * x wu') wd'.

    x (tokens, hidden), wg and wu (inner, hidden), wd (hidden, inner), one type
    act         "silu", "gelu" (by the normal distribution) or "gelu_tanh"
    x_stride    elements between rows of x
    y_stride    elements between rows of y, residual and dy
    """
    _destroy = staticmethod(head_capi.gated_ffn_desc_destroy)

    def __init__(self, tokens, hidden, inner, dtype="bf16", act="silu", x_stride=None, y_stride=None):
        self.tokens, self.hidden, self.inner, self.dtype, self.act = tokens, hidden, inner, dtype, act
        self.x_stride, self.y_stride = x_stride or hidden, y_stride or hidden
        self.desc = head_capi.gated_ffn_desc_create(tokens, hidden, inner, dtype, act)
        if self.x_stride != hidden or self.y_stride != hidden:
            head_capi.gated_ffn_desc_set_row_strides(self.desc, self.x_stride, self.y_stride)
        self.workspace_bytes, self.backward_workspace_bytes, saved = head_capi.gated_ffn_workspace_size(self.desc)
        self._x, self._y = _Rows(tokens, hidden, self.x_stride, dtype), _Rows(tokens, hidden, self.y_stride, dtype)
        self._dx = _Rows(tokens, hidden, hidden, dtype)
        self._wh, self._wd = _Flat((inner, hidden), _TORCH_DTYPE[dtype]), _Flat((hidden, inner), _TORCH_DTYPE[dtype])
        self._saved = _Flat((saved,), torch.uint8)

    def _check(self, x, wg, wu, wd, dev):
        self._x.check("x", x, dev)
        self._wh.check("wg", wg, dev)
        self._wh.check("wu", wu, dev)
        self._wd.check("wd", wd, dev)

    def __call__(self, x, wg, wu, wd, residual=None, y=None, save=False, workspace=None, stream=None):
        """y, or (y, saved) with `save` (what `backward` needs).  y may be residual,
        or x where their strides agree."""
        dev = x.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self(x, wg, wu, wd, residual, y, save, workspace)
        self._check(x, wg, wu, wd, dev)
        if residual is not None:
            self._y.check("residual", residual, dev)
        at = x.device
        if y is None:
            y = self._y.new(at)
        else:
            self._y.check("y", y, dev)
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=at)
        else:
            _check_workspace(workspace, dev)
        saved = self._saved.new(at) if save else None
        head_capi.gated_ffn_fwd(self.desc, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), _ptr(residual),
                                y.data_ptr(), _ptr(saved), workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
        return (y, saved) if save else y

    def backward(self, dy, x, wg, wu, wd, saved, need_dx=True, need_dw=True, workspace=None, stream=None):
        """(dx, dwg, dwu, dwd); None in the place of what is not needed."""
        dev = x.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self.backward(dy, x, wg, wu, wd, saved, need_dx, need_dw, workspace)
        self._check(x, wg, wu, wd, dev)
        self._y.check("dy", dy, dev)
        self._saved.check("saved", saved, dev)
        at = x.device
        if workspace is None:
            workspace = torch.empty(self.backward_workspace_bytes, dtype=torch.uint8, device=at)
        else:
            _check_workspace(workspace, dev)
        dx = self._dx.new(at) if need_dx else None
        dwg, dwu, dwd = (self._wh.new(at), self._wh.new(at), self._wd.new(at)) if need_dw else (None,) * 3
        head_capi.gated_ffn_bwd(self.desc, dy.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(),
                                saved.data_ptr(), _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(dwd), workspace.data_ptr(),
                                workspace.numel(), _raw_stream(dev))
        return dx, dwg, dwu, dwd


AdamWState = collections.namedtuple("AdamWState", "m v m_scale v_scale")


class AdamW(_Op):
    """A step of AdamW over tensors of `sizes` elements at once, in place.

    params fp32, grads of `grad_dtype`, contiguous and of any shape
    states        "f32", or "8bit": moments in 8 bits with a scale for each 256 elements
    copy_dtype    "f16" or "bf16": every step also writes the parameters in that type
    weight_decay  one value, or one for each tensor
    """
    _destroy = staticmethod(head_capi.adamw_desc_destroy)

    def __init__(self, sizes, grad_dtype="f32", states="f32", copy_dtype=None, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.0):
        if copy_dtype not in (None, "f16", "bf16"):
            raise ValueError("copies are f16 or bf16: the parameters are fp32 themselves")
        self.sizes, self.states, self.grad_dtype, self.copy_dtype = tuple(map(int, sizes)), states, grad_dtype, copy_dtype
        self.desc = head_capi.adamw_desc_create(self.sizes, grad_dtype, states, copy_dtype or "f32")
        head_capi.adamw_desc_set_rates(self.desc, *betas, eps)
        decay = [weight_decay] * len(self.sizes) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != len(self.sizes):
            raise ValueError(f"{len(decay)} weight decays for {len(self.sizes)} tensors")
        head_capi.adamw_desc_set_weight_decay(self.desc, decay)
        self.elements = head_capi.adamw_state_elements(self.desc)
        self._grad, self._copy = _TORCH_DTYPE[grad_dtype], _TORCH_DTYPE[copy_dtype] if copy_dtype else None
        kinds = (torch.float32,) * 2 if states == "f32" else (torch.float8_e4m3fn, torch.float8_e5m2)
        self._m, self._v = (_Flat((self.elements,), k) for k in kinds)
        self._scales = _Flat((self.elements // 256,), torch.float8_e8m0fnu)

    def new_state(self, device="cuda"):
        """The moments before the first step.  In 8 bits a value is its code times its block's scale."""
        zeros = [torch.zeros(k.shape, dtype=torch.uint8, device=device).view(k.dtype) if k.dtype.itemsize == 1
                 else torch.zeros(k.shape, dtype=k.dtype, device=device) for k in (self._m, self._v)]
        scales = [torch.zeros(self._scales.shape, dtype=torch.uint8, device=device).view(self._scales.dtype)
                  for _ in range(2)] if self.states != "f32" else [None, None]
        return AdamWState(*zeros, *scales)

    def offset(self, i):
        """Where the moments of tensor i begin."""
        return head_capi.adamw_state_offset(self.desc, i)

    def _addresses(self, name, tensors, dtype, dev):
        if len(tensors) != len(self.sizes):
            raise ValueError(f"{len(tensors)} {name} for {len(self.sizes)} tensors")
        # (A method at a time over all tensors: a loop over tensors takes a third longer.)
        if tuple(map(torch.Tensor.numel, tensors)) != self.sizes or not all(map(torch.Tensor.is_contiguous, tensors)) \
                or (set(map(torch.Tensor.get_device, tensors)) | {dev}) != {dev} \
                or (set(map(_dtype_of, tensors)) | {dtype}) != {dtype}:
            raise ValueError(f"{name} must be contiguous CUDA tensors of {dtype} and of the operator's sizes, on the "
                             f"device of the state")
        return list(map(torch.Tensor.data_ptr, tensors))

    def __call__(self, params, grads, state, step, lr, copies=None, grad_scale=None, skip=None, seed=0, stream=None):
        """Step number `step` (from 1 on).  step and lr are numbers, or tensors of one
        element on the GPU (int64, fp32) that a captured call reads when it runs.
        grad_scale and skip: None or such an fp32 tensor; unless skip holds zero,
        nothing changes.  `seed` draws the roundings of 8-bit states."""
        dev = state.m.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            with _place(dev, stream):
                return self(params, grads, state, step, lr, copies, grad_scale, skip, seed)
        self._m.check("state.m", state.m, dev)
        self._v.check("state.v", state.v, dev)
        ms = vs = 0
        if self.states != "f32":
            if state.m_scale is None or state.v_scale is None:
                raise ValueError("8-bit moments need their scales")
            self._scales.check("state.m_scale", state.m_scale, dev)
            self._scales.check("state.v_scale", state.v_scale, dev)
            ms, vs = state.m_scale.data_ptr(), state.v_scale.data_ptr()
        p = self._addresses("params", params, torch.float32, dev)
        g = self._addresses("grads", grads, self._grad, dev)
        if (copies is None) != (self._copy is None):
            raise ValueError("copies are given where the operator was made with a copy_dtype, and only there")
        c = self._addresses("copies", copies, self._copy, dev) if copies is not None else None
        for name, a in (("params", p), ("copies", c)):
            # (Empty tensors may share an address.)
            if a is not None and len(set(a)) != len(a) \
                    and len(set(k for k, n in zip(a, self.sizes) if n)) != sum(n > 0 for n in self.sizes):
                raise ValueError(f"a tensor is among {name} twice")
        at = []
        for name, t, dtype in (("step", step, torch.int64), ("lr", lr, torch.float32),
                               ("grad_scale", grad_scale, torch.float32), ("skip", skip, torch.float32)):
            if isinstance(t, torch.Tensor):
                if t.dtype is not dtype or t.numel() != 1 or t.get_device() != dev:
                    raise ValueError(f"{name} must be a CUDA tensor of {dtype} and one element, on the device of the state")
                at.append(t.data_ptr())
            else:
                at.append(0)
        if (grad_scale is not None and not at[2]) or (skip is not None and not at[3]):
            raise ValueError("grad_scale and skip are tensors or None")
        head_capi.adamw_step(self.desc, p, g, c, state.m.data_ptr(), state.v.data_ptr(), ms, vs, 0 if at[0] else step,
                             0.0 if at[1] else lr, *at, seed, _raw_stream(dev))


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
