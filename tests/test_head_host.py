"""Host-side checks of the training-head operators' C ABI (include/head.h):
exports, descriptor and argument refusals, workspace sizes.  No kernel is
launched here; the pointers are fake addresses that every call refuses or
ignores before it touches a device."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                  # an aligned address


@pytest.fixture(scope="module")
def capi():
    from dense_convolution_gb300 import build, capi
    build.build()
    return capi


@pytest.fixture(scope="module")
def head(capi):
    from dense_convolution_gb300 import head_capi
    head_capi.load()
    return head_capi


def _status(capi, f, *args):
    try:
        f(*args)
    except capi.Conv2dError as e:
        return e.status
    return capi.OK


def test_exports_every_declared_symbol(capi, head):
    src = open(os.path.join(ROOT, "include", "head.h")).read()
    names = set(re.findall(r"\bconv2d_status ([a-z_]+)\(", src))
    assert names == set(head.EXPORTED) and len(head.EXPORTED) == len(names)
    lib = ctypes.CDLL(capi.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("args", [(-1, 8), (4, 0), (4, -3), (1 << 31, 8), (4, 1 << 31)])
def test_bad_sizes(capi, head, args):
    assert _status(capi, head.layernorm_desc_create, *args) == capi.ERR_BAD_PARAM
    assert _status(capi, head.dropout_desc_create, *args) == capi.ERR_BAD_PARAM


@pytest.mark.parametrize("eps", [-1e-5, float("nan"), float("inf")])
def test_layernorm_bad_eps(capi, head, eps):
    assert _status(capi, head.layernorm_desc_create, 4, 8, "f32", "f32", eps) == capi.ERR_BAD_PARAM


def test_layernorm_types(capi, head):
    for dt, pt, ok in (("f32", "f32", True), ("f16", "f32", True), ("bf16", "bf16", True), ("f32", "f16", False),
                       ("f16", "bf16", False), ("f32", 7, False), (9, "f32", False)):
        try:
            d = head.layernorm_desc_create(4, 8, dt, pt)
        except capi.Conv2dError as e:
            assert not ok and e.status == capi.ERR_BAD_PARAM
        else:
            assert ok, (dt, pt)
            head.layernorm_desc_destroy(d)


def test_layernorm_layouts(capi, head):
    d = head.layernorm_desc_create(12, 8)
    assert _status(capi, head.layernorm_desc_set_row_strides, d, 7, 8) == capi.ERR_BAD_PARAM
    assert _status(capi, head.layernorm_desc_set_row_strides, d, 8, 7) == capi.ERR_BAD_PARAM
    assert _status(capi, head.layernorm_desc_set_planes, d, 5) == capi.ERR_BAD_PARAM
    assert _status(capi, head.layernorm_desc_set_planes, d, -1) == capi.ERR_BAD_PARAM
    head.layernorm_desc_set_planes(d, 6)
    assert _status(capi, head.layernorm_desc_set_row_strides, d, 9, 8) == capi.ERR_UNSUPPORTED
    head.layernorm_desc_set_row_strides(d, 8, 11)
    head.layernorm_desc_set_planes(d, 0)
    head.layernorm_desc_set_row_strides(d, 9, 8)
    assert _status(capi, head.layernorm_desc_set_planes, d, 6) == capi.ERR_UNSUPPORTED
    head.layernorm_desc_destroy(d)
    d = head.layernorm_desc_create(4, 16385)
    assert _status(capi, head.layernorm_desc_set_planes, d, 4) == capi.ERR_UNSUPPORTED
    head.layernorm_desc_destroy(d)


def test_layernorm_arguments(capi, head):
    d = head.layernorm_desc_create(4, 8, "f16", "f32")
    ws = head.layernorm_workspace_size(d)
    assert ws > 0
    fwd = lambda **k: _status(capi, head.layernorm_fwd, d, *{**dict(x=A, gamma=A, beta=A, y=A, mean=A, rstd=A), **k}.values())
    for k, v, want in (("x", 0, capi.ERR_NULL_PTR), ("y", 0, capi.ERR_NULL_PTR), ("x", A + 1, capi.ERR_MISALIGNED),
                       ("y", A + 1, capi.ERR_MISALIGNED), ("gamma", A + 2, capi.ERR_MISALIGNED),
                       ("beta", A + 2, capi.ERR_MISALIGNED), ("mean", A + 2, capi.ERR_MISALIGNED),
                       ("rstd", A + 1, capi.ERR_MISALIGNED)):
        assert fwd(**{k: v}) == want, k
    base = dict(dy=A, x=A, gamma=A, mean=A, rstd=A, dx=A, dgamma=A, dbeta=A, ws=A, bytes=ws)
    bwd = lambda **k: _status(capi, head.layernorm_bwd, d, *{**base, **k}.values())
    for k, v, want in (("dy", 0, capi.ERR_NULL_PTR), ("x", 0, capi.ERR_NULL_PTR), ("mean", 0, capi.ERR_NULL_PTR),
                       ("rstd", 0, capi.ERR_NULL_PTR), ("ws", 0, capi.ERR_NULL_PTR), ("ws", A + 8, capi.ERR_MISALIGNED),
                       ("dx", A + 1, capi.ERR_MISALIGNED), ("dgamma", A + 2, capi.ERR_MISALIGNED),
                       ("dbeta", A + 2, capi.ERR_MISALIGNED), ("bytes", ws - 1, capi.ERR_WORKSPACE_TOO_SMALL)):
        assert bwd(**{k: v}) == want, k
    assert bwd(dx=0, dgamma=0, dbeta=0) == capi.OK             # nothing wanted, nothing launched
    assert _status(capi, head.layernorm_fwd, 0, A, A, A, A) == capi.ERR_NULL_PTR
    head.layernorm_desc_destroy(d)
    d = head.layernorm_desc_create(0, 8)
    assert _status(capi, head.layernorm_fwd, d, 0, 0, 0, 0) == capi.OK     # no rows
    head.layernorm_desc_destroy(d)


@pytest.mark.parametrize("p", [-0.1, 1.1, float("nan")])
def test_dropout_bad_probability(capi, head, p):
    assert _status(capi, head.dropout_desc_create, 4, 8, "f32", p) == capi.ERR_BAD_PARAM


def test_dropout_arguments(capi, head):
    d = head.dropout_desc_create(4, 8, "bf16", 0.5)
    assert _status(capi, head.dropout_desc_set_row_strides, d, 7, 8, 8) == capi.ERR_BAD_PARAM
    assert _status(capi, head.dropout_desc_set_row_strides, d, 8, 7, 8) == capi.ERR_BAD_PARAM
    assert _status(capi, head.dropout_desc_set_row_strides, d, 8, 8, 7) == capi.ERR_BAD_PARAM
    assert _status(capi, head.dropout_fwd, d, 0, 0, A, 1, 0) == capi.ERR_NULL_PTR
    assert _status(capi, head.dropout_fwd, d, A, 0, 0, 1, 0) == capi.ERR_NULL_PTR
    assert _status(capi, head.dropout_fwd, d, A + 1, 0, A, 1, 0) == capi.ERR_MISALIGNED
    assert _status(capi, head.dropout_fwd, d, A, A + 1, A, 1, 0) == capi.ERR_MISALIGNED
    assert _status(capi, head.dropout_fwd, d, A, 0, A, 1, 1 << 63) == capi.ERR_BAD_PARAM
    assert _status(capi, head.dropout_bwd, d, A, 0, 1, 0) == capi.ERR_NULL_PTR
    assert _status(capi, head.dropout_bwd, d, A, A, 1, 1 << 63) == capi.ERR_BAD_PARAM
    head.dropout_desc_destroy(d)


@pytest.mark.parametrize("args", [(-1, 8, 8), (4, 0, 8), (4, 8, 0), (1 << 31, 8, 8), (4, 1 << 27, 8), (4, 8, 1 << 31),
                                  (1 << 30, 8, 1 << 30)])
def test_linear_ce_bad_sizes(capi, head, args):
    assert _status(capi, head.linear_ce_desc_create, *args) == capi.ERR_BAD_PARAM


def test_linear_ce_arguments(capi, head):
    assert _status(capi, head.linear_ce_desc_create, 4, 8, 8, "bf16", 3) == capi.ERR_BAD_PARAM
    assert _status(capi, head.linear_ce_desc_create, 4, 8, 8, 5, "mean") == capi.ERR_BAD_PARAM
    d = head.linear_ce_desc_create(4, 16, 100)
    assert _status(capi, head.linear_ce_desc_set_row_strides, d, 15, 16) == capi.ERR_BAD_PARAM
    assert _status(capi, head.linear_ce_desc_set_row_strides, d, 16, 15) == capi.ERR_BAD_PARAM
    assert _status(capi, head.linear_ce_desc_set_piece, d, -1) == capi.ERR_BAD_PARAM
    f, b = head.linear_ce_workspace_size(d)
    base = dict(h=A, w=A, target=A, loss=A, lse=A, ws=A, bytes=f)
    fwd = lambda **k: _status(capi, head.linear_ce_fwd, d, *{**base, **k}.values())
    for k in ("h", "w", "target", "loss", "lse", "ws"):
        assert fwd(**{k: 0}) == capi.ERR_NULL_PTR, k
    for k, off in (("h", 8), ("w", 2), ("target", 4), ("loss", 2), ("lse", 1), ("ws", 8)):
        assert fwd(**{k: A + off}) == capi.ERR_MISALIGNED, k
    assert fwd(bytes=f - 1) == capi.ERR_WORKSPACE_TOO_SMALL
    base = dict(h=A, w=A, target=A, lse=A, dloss=A, dh=A, dw=A, ws=A, bytes=b)
    bwd = lambda **k: _status(capi, head.linear_ce_bwd, d, *{**base, **k}.values())
    for k in ("h", "w", "target", "lse", "dloss", "ws"):
        assert bwd(**{k: 0}) == capi.ERR_NULL_PTR, k
    for k, off in (("h", 8), ("w", 2), ("target", 4), ("lse", 2), ("dloss", 1), ("dh", 1), ("dw", 1), ("ws", 8)):
        assert bwd(**{k: A + off}) == capi.ERR_MISALIGNED, k
    assert bwd(bytes=b - 1) == capi.ERR_WORKSPACE_TOO_SMALL
    assert bwd(dh=0, dw=0) == capi.OK
    head.linear_ce_desc_destroy(d)


def test_linear_ce_packed_operands_need_element_alignment_only(capi, head):
    d = head.linear_ce_desc_create(4, 15, 100, "f16")          # rows off the 16-byte boundary: copied first
    f, _ = head.linear_ce_workspace_size(d)
    assert _status(capi, head.linear_ce_fwd, d, A + 1, A, A, A, A, A, f) == capi.ERR_MISALIGNED
    assert _status(capi, head.linear_ce_fwd, d, A + 2, A + 2, A, A, A, A, f - 1) == capi.ERR_WORKSPACE_TOO_SMALL
    head.linear_ce_desc_destroy(d)


def test_linear_ce_workspace_follows_the_piece(capi, head):
    d = head.linear_ce_desc_create(1024, 512, 32768, "bf16")
    _, whole = head.linear_ce_workspace_size(d)
    head.linear_ce_desc_set_piece(d, 1024)
    _, piece = head.linear_ce_workspace_size(d)
    assert piece < whole
    assert piece >= 1024 * 1024 * 2                             # dz of one piece
    head.linear_ce_desc_set_piece(d, 0)
    assert head.linear_ce_workspace_size(d)[1] == whole
    head.linear_ce_desc_destroy(d)
