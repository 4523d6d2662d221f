"""Host-side checks of the feed-forward block's C ABI (include/head.h): descriptor and
argument refusals, workspace sizes.  No kernel is launched here; the pointers are
fake addresses that every call refuses or ignores before it touches a device."""
import ctypes

import pytest

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


@pytest.mark.parametrize("args", [(-1, 8, 8), (4, 0, 8), (4, 8, 0), ((1 << 30) + 1, 8, 8), (4, 16385, 8), (4, 8, (1 << 20) + 1),
                                  (1 << 30, 8, 1 << 20), (4, 8, 8, 9), (4, 8, 8, "f16", 3), (4, 8, 8, "f16", -1)])
def test_bad_problems(capi, head, args):
    assert _status(capi, head.gated_ffn_desc_create, *args) == capi.ERR_BAD_PARAM


def test_null_descriptors(capi, head):
    L = head.load()
    assert L.gated_ffn_desc_create(None, 4, 8, 8, 0, 0) == capi.ERR_NULL_PTR
    assert L.gated_ffn_desc_set_row_strides(None, 8, 8) == capi.ERR_NULL_PTR
    assert L.gated_ffn_workspace_size(None, None, None, None) == capi.ERR_NULL_PTR
    assert L.gated_ffn_desc_destroy(None) == capi.OK


def test_strides_and_sizes(capi, head):
    d = head.gated_ffn_desc_create(100, 64, 200, "bf16")
    for xs, ys in ((63, 64), (64, 63), (1 << 39, 64), (64, 1 << 39)):
        assert _status(capi, head.gated_ffn_desc_set_row_strides, d, xs, ys) == capi.ERR_BAD_PARAM
    f, b, s = head.gated_ffn_workspace_size(d)
    assert s == 128 * 2 * 256 * 4 + 100 * 256 * 2 and f >= 100 * 256 * 2 and b >= 2 * 100 * 256 * 2
    head.gated_ffn_desc_set_row_strides(d, 67, 65)                # both are copied now
    f2, b2, s2 = head.gated_ffn_workspace_size(d)
    assert f2 >= f + 100 * 64 * 2 and b2 >= b + 2 * 100 * 64 * 2 and s2 == s
    one = ctypes.c_size_t()
    assert head.load().gated_ffn_workspace_size(d, None, None, ctypes.byref(one)) == capi.OK and one.value == s
    head.gated_ffn_desc_destroy(d)


@pytest.mark.parametrize("tokens", [1, 300])
@pytest.mark.parametrize("dtype,hidden,inner", [("bf16", 64, 128), ("f16", 60, 100), ("f32", 64, 128)])
def test_arguments(capi, head, tokens, dtype, hidden, inner):
    e = 4 if dtype == "f32" else 2
    free = dtype == "f32"                                       # operands that are copied need their element's alignment
    d = head.gated_ffn_desc_create(tokens, hidden, inner, dtype)
    f, b, _ = head.gated_ffn_workspace_size(d)
    base = dict(x=A, wg=A, wu=A, wd=A, res=A, y=A, saved=A, ws=A, bytes=f)
    fwd = lambda **k: _status(capi, head.gated_ffn_fwd, d, *{**base, **k}.values())
    for k in ("x", "wg", "wu", "wd", "y", "ws"):
        assert fwd(**{k: 0}) == capi.ERR_NULL_PTR, k
    in_place = {"x": hidden % 8 == 0, "wg": hidden % 8 == 0, "wu": hidden % 8 == 0, "wd": inner % 8 == 0}
    for k, v in in_place.items():
        assert fwd(**{k: A + 1}) == capi.ERR_MISALIGNED, k
        want = capi.ERR_MISALIGNED if v and not free else capi.ERR_WORKSPACE_TOO_SMALL
        assert fwd(**{k: A + e, "bytes": f - 1}) == want, k
    for k, off in (("res", 1), ("y", 1), ("saved", 16), ("ws", 8)):
        assert fwd(**{k: A + off}) == capi.ERR_MISALIGNED, k
    assert fwd(bytes=f - 1) == capi.ERR_WORKSPACE_TOO_SMALL
    base = dict(dy=A, x=A, wg=A, wu=A, wd=A, saved=A, dx=A, dwg=A, dwu=A, dwd=A, ws=A, bytes=b)
    bwd = lambda **k: _status(capi, head.gated_ffn_bwd, d, *{**base, **k}.values())
    for k in ("dy", "x", "wg", "wu", "wd", "saved", "ws"):
        assert bwd(**{k: 0}) == capi.ERR_NULL_PTR, k
    for k, off in (("dy", 1), ("x", 1), ("wg", 1), ("wu", 1), ("wd", 1), ("saved", 16), ("dx", 1), ("dwg", 1), ("dwu", 1),
                   ("dwd", 1), ("ws", 8)):
        assert bwd(**{k: A + off}) == capi.ERR_MISALIGNED, k
    assert bwd(bytes=b - 1) == capi.ERR_WORKSPACE_TOO_SMALL
    assert bwd(dx=0, dwg=0, dwu=0, dwd=0) == capi.OK             # nothing wanted, nothing launched
    assert _status(capi, head.gated_ffn_fwd, 0, *{**dict(x=A, wg=A, wu=A, wd=A, res=A, y=A, saved=A, ws=A, bytes=f)}.values()) == capi.ERR_NULL_PTR
    head.gated_ffn_desc_destroy(d)


def test_no_tokens(capi, head):
    d = head.gated_ffn_desc_create(0, 8, 8)
    assert _status(capi, head.gated_ffn_fwd, d, 0, 0, 0, 0, 0, 0, 0, 0, 0) == capi.OK
    head.gated_ffn_desc_destroy(d)
