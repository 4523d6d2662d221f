"""ctypes binding of ``include/head.h`` — argument marshalling only.

The training-head operators live in the same shared library as the
convolution and follow ``capi``'s conventions: each function has the name of
the C entry point it wraps, raises ``Conv2dError`` on a non-OK status, and takes
pointers (device addresses) and streams as plain integers, 0 for none (NULL).
"""
from __future__ import annotations

import ctypes

from . import capi
from .capi import DTYPES, _check

REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}

EXPORTED = ("layernorm_desc_create", "layernorm_desc_set_row_strides", "layernorm_desc_set_planes",
            "layernorm_desc_destroy", "layernorm_workspace_size", "layernorm_fwd", "layernorm_bwd",
            "dropout_desc_create", "dropout_desc_set_row_strides", "dropout_desc_destroy", "dropout_fwd", "dropout_bwd",
            "linear_ce_desc_create", "linear_ce_desc_set_row_strides", "linear_ce_desc_set_piece",
            "linear_ce_desc_set_dz_parts", "linear_ce_desc_destroy", "linear_ce_workspace_size", "linear_ce_fwd", "linear_ce_bwd")

_lib = None


def load():
    """The shared library with the head's signatures set (once)."""
    global _lib
    if _lib is not None:
        return _lib
    L = capi.load()
    i32, i64, u64, size, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_void_p
    out = ctypes.POINTER(vp)
    L.layernorm_desc_create.argtypes = [out, i64, i64, i32, i32, ctypes.c_float]
    L.layernorm_desc_set_row_strides.argtypes = [vp, i64, i64]
    L.layernorm_desc_set_planes.argtypes = [vp, i64]
    L.layernorm_desc_destroy.argtypes = [vp]
    L.layernorm_workspace_size.argtypes = [vp, ctypes.POINTER(size)]
    L.layernorm_fwd.argtypes = [vp] * 8
    L.layernorm_bwd.argtypes = [vp] * 10 + [size, vp]
    L.dropout_desc_create.argtypes = [out, i64, i64, i32, ctypes.c_double]
    L.dropout_desc_set_row_strides.argtypes = [vp, i64, i64, i64]
    L.dropout_desc_destroy.argtypes = [vp]
    L.dropout_fwd.argtypes = [vp, vp, vp, vp, u64, u64, vp]
    L.dropout_bwd.argtypes = [vp, vp, vp, u64, u64, vp]
    L.linear_ce_desc_create.argtypes = [out, i64, i64, i64, i32, i32, i64]
    L.linear_ce_desc_set_row_strides.argtypes = [vp, i64, i64]
    L.linear_ce_desc_set_piece.argtypes = [vp, i64]
    L.linear_ce_desc_set_dz_parts.argtypes = [vp, i32]
    L.linear_ce_desc_destroy.argtypes = [vp]
    L.linear_ce_workspace_size.argtypes = [vp, ctypes.POINTER(size), ctypes.POINTER(size)]
    L.linear_ce_fwd.argtypes = [vp] * 7 + [size, vp]
    L.linear_ce_bwd.argtypes = [vp] * 9 + [size, vp]
    for f in EXPORTED:
        getattr(L, f).restype = i32
    _lib = L
    return L


def _dtype(t):
    return DTYPES[t] if isinstance(t, str) else int(t)


def layernorm_desc_create(rows, cols, dtype="f32", param_dtype="f32", eps=1e-5) -> int:
    d = ctypes.c_void_p()
    _check(load().layernorm_desc_create(ctypes.byref(d), rows, cols, _dtype(dtype), _dtype(param_dtype), eps),
           "layernorm_desc_create")
    return d.value


def layernorm_desc_set_row_strides(desc: int, x_stride: int, y_stride: int):
    _check(load().layernorm_desc_set_row_strides(desc, x_stride, y_stride), "layernorm_desc_set_row_strides")


def layernorm_desc_set_planes(desc: int, pixels: int):
    _check(load().layernorm_desc_set_planes(desc, pixels), "layernorm_desc_set_planes")


def layernorm_desc_destroy(desc: int):
    _check(load().layernorm_desc_destroy(desc), "layernorm_desc_destroy")


def layernorm_workspace_size(desc: int) -> int:
    b = ctypes.c_size_t()
    _check(load().layernorm_workspace_size(desc, ctypes.byref(b)), "layernorm_workspace_size")
    return b.value


def layernorm_fwd(desc: int, x: int, gamma: int, beta: int, y: int, mean: int = 0, rstd: int = 0, stream: int = 0):
    s = load().layernorm_fwd(desc, x, gamma, beta, y, mean, rstd, stream)
    if s:
        _check(s, "layernorm_fwd")


def layernorm_bwd(desc: int, dy: int, x: int, gamma: int, mean: int, rstd: int, dx: int, dgamma: int, dbeta: int,
                  workspace: int, workspace_bytes: int, stream: int = 0):
    _check(load().layernorm_bwd(desc, dy, x, gamma, mean, rstd, dx,
                                dgamma, dbeta, workspace, workspace_bytes, stream),
           "layernorm_bwd")


def dropout_desc_create(rows, cols, dtype="f32", p=0.5) -> int:
    d = ctypes.c_void_p()
    _check(load().dropout_desc_create(ctypes.byref(d), rows, cols, _dtype(dtype), p), "dropout_desc_create")
    return d.value


def dropout_desc_set_row_strides(desc: int, x_stride: int, residual_stride: int, y_stride: int):
    _check(load().dropout_desc_set_row_strides(desc, x_stride, residual_stride, y_stride),
           "dropout_desc_set_row_strides")


def dropout_desc_destroy(desc: int):
    _check(load().dropout_desc_destroy(desc), "dropout_desc_destroy")


def dropout_fwd(desc: int, x: int, residual: int, y: int, seed: int, offset: int, stream: int = 0):
    _check(load().dropout_fwd(desc, x, residual, y, seed, offset, stream),
           "dropout_fwd")


def dropout_bwd(desc: int, dy: int, dx: int, seed: int, offset: int, stream: int = 0):
    _check(load().dropout_bwd(desc, dy, dx, seed, offset, stream), "dropout_bwd")


def linear_ce_desc_create(tokens, hidden, vocab, dtype="bf16", reduction="mean", ignore_index=-100) -> int:
    d = ctypes.c_void_p()
    red = REDUCTIONS[reduction] if isinstance(reduction, str) else int(reduction)
    _check(load().linear_ce_desc_create(ctypes.byref(d), tokens, hidden, vocab, _dtype(dtype), red, ignore_index),
           "linear_ce_desc_create")
    return d.value


def linear_ce_desc_set_row_strides(desc: int, h_stride: int, w_stride: int):
    _check(load().linear_ce_desc_set_row_strides(desc, h_stride, w_stride), "linear_ce_desc_set_row_strides")


def linear_ce_desc_set_piece(desc: int, vocab_rows: int):
    _check(load().linear_ce_desc_set_piece(desc, vocab_rows), "linear_ce_desc_set_piece")


def linear_ce_desc_set_dz_parts(desc: int, parts: int):
    _check(load().linear_ce_desc_set_dz_parts(desc, parts), "linear_ce_desc_set_dz_parts")


def linear_ce_desc_destroy(desc: int):
    _check(load().linear_ce_desc_destroy(desc), "linear_ce_desc_destroy")


def linear_ce_workspace_size(desc: int):
    """Workspace bytes of (linear_ce_fwd, linear_ce_bwd)."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().linear_ce_workspace_size(desc, ctypes.byref(f), ctypes.byref(b)), "linear_ce_workspace_size")
    return f.value, b.value


def linear_ce_fwd(desc: int, h: int, w: int, target: int, loss: int, lse: int, workspace: int, workspace_bytes: int,
                  stream: int = 0):
    _check(load().linear_ce_fwd(desc, h, w, target, loss, lse,
                                workspace, workspace_bytes, stream), "linear_ce_fwd")


def linear_ce_bwd(desc: int, h: int, w: int, target: int, lse: int, dloss: int, dh: int, dw: int, workspace: int,
                  workspace_bytes: int, stream: int = 0):
    _check(load().linear_ce_bwd(desc, h, w, target, lse, dloss, dh,
                                dw, workspace, workspace_bytes, stream), "linear_ce_bwd")
