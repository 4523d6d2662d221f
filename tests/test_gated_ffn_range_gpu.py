"""fp16 gradients of the feed-forward block whose dg and du are far from dy: held as fp16 numbers on
a scale of their own, they keep their digits.

A row's own digits: dg, du and the result round by 0.43 u in the mean, together 0.6 u in the
2-norm.  A row's 2-norm over some 256 results, the large ones counting most, strays by a fourteenth, and the worst of
300 rows by three times that: 0.73 u, and 0.85 u is allowed.
"""
import pytest

from .test_gated_ffn_gpu import U, _inputs, _lib, _reference, _run, _status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [40, 300])
def test_rows_that_are_not_finite_leave_the_others_their_digits(t):
    """The scale goes by the finite values: du of some 2^-17 keeps its digits beside a row of NaN."""
    import torch
    from dense_convolution_gb300 import head
    d, f = 256, 512
    i = _inputs(23, t, d, f, "f16", dy_scale=2.0 ** -17)
    i["wu"] *= 2.0 ** 8
    want = _reference(i, "silu", "f16")
    i["dy"][5], i["dy"][7, 3], i["x"][11, 2] = float("nan"), float("inf"), float("inf")
    got = _run(head.GatedFeedForward(t, d, f, "f16", "silu"), i, need_dw=False)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[[5, 7, 11]] = False
    v = want["dx"][0][keep]
    off = ((got["dx"][keep].double() - v).norm(dim=1) / v.norm(dim=1)).max()
    assert float(off) <= 0.85 * U["f16"], float(off) / U["f16"]
    assert not torch.isfinite(got["dx"][~keep]).all(dim=1).any()
