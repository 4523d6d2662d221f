"""Host-side checks of AdamW's C ABI (include/head.h): descriptor and argument
refusals, the layout of the moments.  No kernel is launched here; the pointers are
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


def _status(capi, f, *args, **more):
    try:
        f(*args, **more)
    except capi.Conv2dError as e:
        return e.status
    return capi.OK


@pytest.mark.parametrize("sizes", [[-1], [4, -3], [(1 << 34) + 1], [1 << 34] * 64])
def test_bad_sizes(capi, head, sizes):
    assert _status(capi, head.adamw_desc_create, sizes) == capi.ERR_BAD_PARAM


def test_bad_types(capi, head):
    for args in ((9, "f32", "f32"), ("f32", 2, "f32"), ("f32", "f32", 7)):
        assert _status(capi, head.adamw_desc_create, [4], *args) == capi.ERR_BAD_PARAM, args
    L = head.load()
    out = ctypes.c_void_p(5)
    assert L.adamw_desc_create(None, 0, None, 0, 0, 0) == capi.ERR_NULL_PTR
    assert L.adamw_desc_create(ctypes.byref(out), 2, None, 0, 0, 0) == capi.ERR_NULL_PTR and not out.value
    assert L.adamw_desc_create(ctypes.byref(out), -1, None, 0, 0, 0) == capi.ERR_BAD_PARAM
    assert L.adamw_desc_create(ctypes.byref(out), (1 << 24) + 1, None, 0, 0, 0) == capi.ERR_BAD_PARAM


@pytest.mark.parametrize("rates", [(1.0, 0.9, 1e-8), (-0.1, 0.9, 1e-8), (0.9, 1.0, 1e-8), (0.9, float("nan"), 1e-8),
                                   (0.9, 1 - 1e-9, 1e-8), (0.9, 0.99, 0.0), (0.9, 0.99, -1e-8), (0.9, 0.99, 1e-60),
                                   (0.9, 0.99, float("inf")), (0.9, 0.99, float("nan"))])
def test_bad_rates(capi, head, rates):
    d = head.adamw_desc_create([4])
    assert _status(capi, head.adamw_desc_set_rates, d, *rates) == capi.ERR_BAD_PARAM
    head.adamw_desc_set_rates(d, 0.0, 0.0, 1e-30)
    head.adamw_desc_destroy(d)


def test_layout_and_decay(capi, head):
    d = head.adamw_desc_create([1, 0, 256, 257, 1000])
    assert head.adamw_state_elements(d) == 256 + 0 + 256 + 512 + 1024
    assert [head.adamw_state_offset(d, i) for i in range(5)] == [0, 256, 256, 512, 1024]
    for i in (-1, 5):
        assert _status(capi, head.adamw_state_offset, d, i) == capi.ERR_BAD_PARAM
    head.adamw_desc_set_weight_decay(d, [0.0, 0.1, 0.1, 0.0, 1.0])
    assert _status(capi, head.adamw_desc_set_weight_decay, d, [0.0, 0.1, float("nan"), 0.0, 1.0]) == capi.ERR_BAD_PARAM
    assert head.load().adamw_desc_set_weight_decay(d, None) == capi.ERR_NULL_PTR
    head.adamw_desc_destroy(d)
    assert _status(capi, head.adamw_state_elements, 0) == capi.ERR_NULL_PTR


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_step_arguments(capi, head, states):
    d = head.adamw_desc_create([3, 0, 5], "f16", states, "bf16")
    base = dict(params=[A, 0, A], grads=[A, 0, A], copies=[A, 0, A], m=A, v=A, m_scale=A, v_scale=A, step=1, lr=1e-3)
    step = lambda **k: _status(capi, head.adamw_step, d, **{**base, **k})
    for k in ("m", "v") + (("m_scale", "v_scale") if states == "8bit" else ()):
        assert step(**{k: 0}) == capi.ERR_NULL_PTR, k
    for k in ("params", "grads", "copies"):
        assert step(**{k: [A, 0, 0]}) == capi.ERR_NULL_PTR, k
        assert step(**{k: [A, 0, A + 1]}) == capi.ERR_MISALIGNED, k
    assert step(copies=None) == capi.ERR_NULL_PTR
    assert step(params=[A + 2, 0, A]) == capi.ERR_MISALIGNED
    for k in ("m", "v"):
        assert step(**{k: A + 16}) == capi.ERR_MISALIGNED, k
    for k, off in (("device_step", 4), ("device_lr", 2), ("grad_scale", 1), ("skip", 2)):
        assert step(**{k: A + off}) == capi.ERR_MISALIGNED, k
    for k, v in (("step", 0), ("step", -1), ("lr", float("nan")), ("lr", float("inf"))):
        assert step(**{k: v}) == capi.ERR_BAD_PARAM, (k, v)
    assert _status(capi, head.adamw_step, 0, **base) == capi.ERR_NULL_PTR
    head.adamw_desc_destroy(d)
    d = head.adamw_desc_create([0, 0])                          # nothing to do
    assert _status(capi, head.adamw_step, d, [0, 0], [0, 0], None, 0, 0) == capi.OK
    head.adamw_desc_destroy(d)
    d = head.adamw_desc_create([])
    assert head.adamw_state_elements(d) == 0 and _status(capi, head.adamw_step, d, [], [], None, 0, 0) == capi.OK
    head.adamw_desc_destroy(d)
