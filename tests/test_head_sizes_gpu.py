"""Sizes at the far end of what a descriptor takes, and sizes that change the form
in which a call runs."""
import pytest

from .test_head_gpu import (E, U, _ce_inputs, _check_ce, _close, _dt, _gen, _lib, _randn, _status,  # noqa: F401
                            _strided)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n,d,v", [("f32", 16, 16, 40_000_000), ("bf16", 3, 8, 2 ** 27 + 2 ** 17 + 5),
                                         ("f16", 2, 5, 2 ** 28 + 77), ("f32", 1, 3, 3_000_001)])
def test_few_tokens_of_a_very_large_vocabulary(dtype, n, d, v):
    """dh in more shares of the vocabulary than a grid's second dimension numbers.
    All rows of w are zero but for the first and the last three."""
    import torch
    from dense_convolution_gb300 import head
    k = 3
    g = _gen(n)
    ends = _randn(g, 2 * k, d).to(_dt(dtype))
    w = torch.zeros(v, d, device="cuda", dtype=_dt(dtype))
    w[:k], w[-k:] = ends[:k], ends[k:]
    h = _randn(g, n, d).to(_dt(dtype))
    target = torch.full((n,), v - 1, device="cuda")
    target[0] = 1
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum")
    loss, lse = op(h, w, target)
    dh, dw = op.backward(h, w, target, lse, torch.ones((), device="cuda"))
    z = h.double() @ ends.double().T
    want = torch.log((v - 2 * k) + z.exp().sum(1))
    # Sums of v ones: exact below 2^24, then joined by a few hundred additions.
    _close(lse, want, 512 * E * want.abs(), "lse")
    y = torch.full((n,), 2 * k - 1, device="cuda")
    y[0] = 1
    _close(loss, (want - z.gather(1, y[:, None])[:, 0]).sum(), n * 512 * E * want.abs().max() + 64 * E * z.abs().sum(), "loss")
    p = torch.exp(z - want[:, None])
    p[torch.arange(n, device="cuda"), y] -= 1.0
    dh_want, size = p @ ends.double(), p.abs() @ ends.double().abs()
    _close(dh, dh_want, U[dtype] * dh_want.abs() + 1e-4 * size, "dh")
    dw_want, size = p.T @ h.double(), p.T.abs() @ h.double().abs()
    _close(torch.cat([dw[:k], dw[-k:]]), dw_want, U[dtype] * dw_want.abs() + 1e-4 * size, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,v", [(256, 64640), (40, 2000), (1024, 5003), (1024, 20000), (509, 10007), (2487, 9731), (8, 200001)])
def test_one_token(dtype, d, v):
    """Either number of rows of w a warp takes, at lengths on both sides of the rule."""
    import torch
    from dense_convolution_gb300 import head
    h, w, target = _ce_inputs(d + v, 1, d, v, dtype, ignored=0.0)
    op = head.LinearCrossEntropy(1, d, v, dtype, reduction="none")
    _check_ce(h, w, target, dtype, "none", op, torch.full((1,), 0.7, device="cuda"))


@pytest.mark.parametrize("n,d,v", [(17, 100, 501), (32, 640, 3001), (31, 33, 700), (11, 4096, 900), (20, 3900, 947),
                                   (9, 6144, 333), (25, 3168, 600), (32, 8, 40), (24, 5, 9000)])
def test_fp32_losses_in_groups_of_tokens(n, d, v):
    """The fp32 forward pass of few tokens in two to four groups, targets ignored in
    the last one too, with rows of h that are not adjacent."""
    import torch
    from dense_convolution_gb300 import head
    h, w, target = _ce_inputs(n * 7 + d, n, d, v, "f32")
    target[-2] = -100
    h, _ = _strided(h, d + 3)
    for reduction in ("none", "sum", "mean"):
        op = head.LinearCrossEntropy(n, d, v, "f32", reduction=reduction, h_stride=d + 3)
        dloss = torch.rand(n, device="cuda") + 0.5 if reduction == "none" else torch.full((), 0.7, device="cuda")
        _check_ce(h, w, target, "f32", reduction, op, dloss, reduction + " ")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v", [(1, 60000, 300), (3, 30001, 200), (9, 25600, 130)])
def test_few_tokens_too_long_for_shared_memory(dtype, n, d, v):
    """Few tokens whose h does not fit a block take the tensor cores."""
    import torch
    from dense_convolution_gb300 import head
    h, w, target = _ce_inputs(d, n, d, v, dtype, ignored=0.0)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum")
    _check_ce(h, w, target, dtype, "sum", op, torch.full((), 0.7, device="cuda"))
