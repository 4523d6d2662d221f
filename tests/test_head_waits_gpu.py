"""Waits that run out, kernel by kernel.  With the limit at a nanosecond the ordinary
waits of a call give up: the status after that call alone says so, and under the
default limit the same call is right again."""
import pytest

from .test_head_gpu import _ce_inputs, _gen, _lib, _randn  # noqa: F401

pytestmark = pytest.mark.gpu


def _loss(n, d, v, dtype):
    def make():
        from dense_convolution_gb300 import head
        op = head.LinearCrossEntropy(n, d, v, dtype)
        h, w, target = _ce_inputs(50, n, d, v, dtype)
        return lambda: op(h, w, target)
    return make


def _loss_backward(n, d, v, dtype, **need):
    def make():
        import torch
        from dense_convolution_gb300 import head
        op = head.LinearCrossEntropy(n, d, v, dtype)
        h, w, target = _ce_inputs(50, n, d, v, dtype)
        _, lse = op(h, w, target)
        one = torch.ones((), device="cuda")
        return lambda: [t for t in op.backward(h, w, target, lse, one, **need) if t is not None]
    return make


def _norm(rows, cols, pixels, backward):
    def make():
        import torch
        from dense_convolution_gb300 import head
        shape = (rows // pixels, cols, pixels) if pixels else (rows, cols)
        x = _randn(_gen(2), *shape).to(torch.bfloat16)
        op = head.LayerNorm(rows, cols, "bf16", "f32", pixels=pixels)
        y, mean, rstd = op(x, stats=True)
        return (lambda: list(op.backward(y, x, None, mean, rstd))) if backward else (lambda: [op(x)])
    return make


@pytest.mark.parametrize("make", [
    _loss(600, 1024, 2000, "bf16"), _loss(100, 512, 900, "f16"), _loss(300, 640, 3000, "f32"),
    _loss_backward(600, 1024, 2000, "bf16"), _loss_backward(100, 512, 900, "f16"), _loss_backward(300, 640, 3000, "f32"),
    _loss_backward(600, 2048, 2000, "f16", need_dw=False), _loss_backward(1500, 200, 9000, "bf16", need_dh=False),
    _norm(3200, 256, 400, False), _norm(3200, 256, 400, True), _norm(800, 1000, 200, True)],
    ids=["loss", "loss_one_row_of_tiles", "loss_fp32", "loss_backward", "loss_backward_split", "loss_backward_fp32",
         "promoted_dz", "dw_alone", "planes", "planes_backward", "wide_planes_backward"])
def test_a_wait_that_runs_out_is_reported(make):
    import torch
    from dense_convolution_gb300 import capi
    call = make()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert capi.conv2d_device_status(stream) == 0
    try:
        capi.conv2d_set_wait_limit(1, stream)
        call()
        torch.cuda.synchronize()
        assert capi.conv2d_device_status(stream) != 0
    finally:
        capi.conv2d_set_wait_limit(0, stream)
    assert all(a.equal(b) for a, b in zip(want, call()))
    assert capi.conv2d_device_status(stream) == 0


@pytest.mark.parametrize("cols,backward", [(2048, False), (2048, True), (1096, True), (8192, True)])
def test_rows_under_the_lowest_limit(cols, backward):
    """The row kernels look for a copy once, for up to a time slice of the hardware,
    before the limit counts: a call under the lowest limit returns, right or reported."""
    import torch
    from dense_convolution_gb300 import capi
    call = _norm(4000, cols, None, backward)()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert capi.conv2d_device_status(stream) == 0
    try:
        capi.conv2d_set_wait_limit(1, stream)
        got = call()
        torch.cuda.synchronize()
        assert capi.conv2d_device_status(stream) != 0 or all(a.equal(b) for a, b in zip(want, got))
    finally:
        capi.conv2d_set_wait_limit(0, stream)
    assert all(a.equal(b) for a, b in zip(want, call()))
    assert capi.conv2d_device_status(stream) == 0
