"""Waits that run out, kernel by kernel.  With the limit at a nanosecond the ordinary
waits of a call give up: the status after that call alone says so, and under the
default limit the same call is right again."""
import pytest

from .test_head_gpu import _ce_inputs, _lib  # noqa: F401

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


@pytest.mark.parametrize("make", [
    _loss(600, 1024, 2000, "bf16"), _loss(100, 512, 900, "f16"), _loss(300, 640, 3000, "f32"),
    _loss_backward(600, 1024, 2000, "bf16"), _loss_backward(100, 512, 900, "f16"), _loss_backward(300, 640, 3000, "f32"),
    _loss_backward(600, 2048, 2000, "f16", need_dw=False), _loss_backward(1500, 200, 9000, "bf16", need_dh=False)],
    ids=["loss", "loss_one_row_of_tiles", "loss_fp32", "loss_backward", "loss_backward_split", "loss_backward_fp32",
         "promoted_dz", "dw_alone"])
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
