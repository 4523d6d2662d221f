"""The parts in which the logits' gradient is kept: refusals and sizes (no GPU), and
what the second part leaves of the error of dh and dw."""
import pytest


@pytest.fixture(scope="module")
def head_capi():
    from dense_convolution_gb300 import build, head_capi
    build.build()
    return head_capi


def _status(f, *args):
    from dense_convolution_gb300 import capi
    try:
        f(*args)
    except capi.Conv2dError as e:
        return e.status
    return capi.OK


def test_refusals_and_workspace(head_capi):
    from dense_convolution_gb300 import capi
    d = head_capi.linear_ce_desc_create(1024, 512, 32768, "bf16")
    size = lambda: head_capi.linear_ce_workspace_size(d)[1]
    one = size()
    for parts in (-1, 3):
        assert _status(head_capi.linear_ce_desc_set_dz_parts, d, parts) == capi.ERR_BAD_PARAM
    head_capi.linear_ce_desc_set_dz_parts(d, 2)
    assert size() >= one + 1024 * 32768 * 2
    head_capi.linear_ce_desc_set_dz_parts(d, 1)
    assert size() == one
    head_capi.linear_ce_desc_set_dz_parts(d, 0)
    assert size() == one
    head_capi.linear_ce_desc_destroy(d)
    d = head_capi.linear_ce_desc_create(100, 512, 32768, "f16")            # two parts by themselves
    two = size()
    head_capi.linear_ce_desc_set_dz_parts(d, 1)
    assert size() < two
    head_capi.linear_ce_desc_destroy(d)
    d = head_capi.linear_ce_desc_create(100, 512, 32768, "f32")
    assert _status(head_capi.linear_ce_desc_set_dz_parts, d, 1) == capi.ERR_UNSUPPORTED
    head_capi.linear_ce_desc_set_dz_parts(d, 0)
    head_capi.linear_ce_desc_destroy(d)
    assert _status(head_capi.linear_ce_desc_set_dz_parts, 0, 1) == capi.ERR_NULL_PTR


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,d,v,piece", [(777, 509, 10007, None), (2000, 264, 3000, 1024), (300, 1032, 9000, None)])
def test_two_parts_leave_the_results_own_rounding(head_capi, dtype, n, d, v, piece):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import capi, head
    from .test_head_gpu import _ce_inputs, _ce_reference, _check_ce
    h, w, target = _ce_inputs(n, n, d, v, dtype)
    one = torch.ones((), device="cuda")
    r = _ce_reference(h, w, target, "sum", one)
    off = {}
    for parts in (1, 2):
        op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum", piece=piece, dz_parts=parts)
        _, _, dh, dw = _check_ce(h, w, target, dtype, "sum", op, one, f"{parts} parts ")
        off[parts] = [float((got.double() - r[k]).norm() / r[k].norm()) for got, k in ((dh, "dh"), (dw, "dw"))]
    least = [float((r[k].to(h.dtype).double() - r[k]).norm() / r[k].norm()) for k in ("dh", "dw")]
    # What two parts keep of dz is 2^-16 (bf16) or 2^-22 of it: far below the rounding
    # of the results, as are their sums' truncation and p's error.
    assert all(off[2][i] < 1.01 * least[i] for i in (0, 1)), (off, least)
    assert all(off[2][i] < off[1][i] for i in (0, 1)), (off, least)
    assert capi.conv2d_device_status(0) == 0
