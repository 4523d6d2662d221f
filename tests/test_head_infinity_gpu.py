"""Infinite logits: the log-sum-exp of a row that holds one is infinite, and only a
logit that is no number makes it NaN."""
import pytest

from .test_head_gpu import _ce_inputs, _lib, _status  # noqa: F401

pytestmark = pytest.mark.gpu


# (fp32 past the few tokens' form: its three parts make an infinite factor NaN, as head.h says.)
@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 4), ("f16", 6), ("f32", 8), ("f32", 15), ("bf16", 140), ("f16", 700)])
def test_an_infinite_weight(dtype, n):
    import torch
    from dense_convolution_gb300 import head
    d, v = 136, 900
    h, w, target = _ce_inputs(3, n, d, v, dtype, ignored=0.0)
    w[700, 5] = float("inf")
    sign = torch.tensor([1.0, -1.0, 0.0], device="cuda")[torch.arange(n, device="cuda") % 3]
    h[:, 5] = sign.to(h.dtype)                             # logit 700: +inf, -inf, NaN in turn
    target[target == 700] = 0
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="none")
    loss, lse = op(h, w, target)
    z = h.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    assert (lse[0::3] == float("inf")).all() and torch.isnan(lse[2::3]).all()
    assert (loss[0::3] == float("inf")).all() and torch.isnan(loss[2::3]).all()
    assert torch.allclose(lse[1::3].double(), want[1::3], rtol=1e-5)
    # The softmax of such a row is 0 but for the infinite logit's own, which is NaN.
    dh, dw = op.backward(h, w, target, lse, torch.ones(n, device="cuda"))
    assert torch.isnan(dw[700].float()).any()
    if n == 1:
        dw[700] = 0
        assert torch.isfinite(dw.float()).all()


@pytest.mark.parametrize("dtype,n", [("bf16", 3), ("f32", 20), ("f16", 300)])
def test_rows_of_nothing_but_minus_infinity(dtype, n):
    """Every logit -inf: so is the log-sum-exp; one that is finite: the others add nothing."""
    import torch
    from dense_convolution_gb300 import head
    d, v = 8, 300
    h = torch.zeros(n, d, device="cuda", dtype={"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype])
    h[:, 0] = 1
    w = torch.zeros(v, d, device="cuda", dtype=h.dtype)
    w[:, 0] = float("-inf")
    target = torch.zeros(n, dtype=torch.int64, device="cuda")
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="none")
    assert (op(h, w, target)[1] == float("-inf")).all()
    w[17, 0] = 2.0
    target[:] = 17
    loss, lse = op(h, w, target)
    assert torch.equal(lse, torch.full_like(lse, 2.0)) and not loss.any()
