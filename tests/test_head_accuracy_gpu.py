"""Sums that all go one way.  A result may be off by its own rounding to the output
type, which has no preferred direction; what the sums behind it lose does have
one, and stays well below that rounding whatever their length.

E = 2^-24.  A tensor-core step (16 terms) truncates by less than 2 E of the sum
so far, which is half of the final one on average: E a step.
"""
import math

import pytest

from .test_head_gpu import E, U, _dt, _gen, _lib, _status, _strided, _randn  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


def _positive(seed, n, d, v, dtype, scale):
    """h and w without a negative value, columns of all sizes; target row 0 of w is zero."""
    import torch
    g = _gen(seed)
    col = lambda: torch.exp2(2 * torch.rand(1, d, generator=g, device="cuda") - 1)
    h = ((torch.rand(n, d, generator=g, device="cuda") + 0.5) * col()).to(_dt(dtype))
    w = ((torch.rand(v, d, generator=g, device="cuda") + 0.1) * col() * scale / d).to(_dt(dtype))
    w[0] = 0
    return h, w, torch.zeros(n, dtype=torch.int64, device="cuda")


def _signed_errors(h, w, target, op, rounded=False):
    """Mean signed relative errors of dh and of dw (without the targets' row), and the
    mean logit.  `rounded`: against the sums of dz rounded to the operands' type,
    which has a direction where all of its values lie within one unit in the last place."""
    import torch
    n, v = h.shape[0], w.shape[0]
    _, lse = op(h, w, target)
    dh, dw = op.backward(h, w, target, lse, torch.ones((), device="cuda"))
    hd, wd = h.double(), w.double()
    want_h, want_w, mean = [], torch.zeros_like(wd), 0.0
    for i in range(0, n, 4096):
        z = hd[i:i + 4096] @ wd.T
        mean += float(z.sum()) / (n * v)
        p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        p[:, 0] -= 1.0
        if rounded:
            p = (p * 2.0 ** 14).to(h.dtype).double() * 2.0 ** -14
        want_h.append(p @ wd)
        want_w += p.T @ hd[i:i + 4096]
    want_h = torch.cat(want_h)
    return (float(((dh.double() - want_h) / want_h).mean()), float(((dw.double() - want_w) / want_w)[1:].mean()), mean)


@pytest.mark.parametrize("dtype,n,d,v", [("f16", 300, 4096, 1000), ("f16", 300, 16384, 1000), ("f16", 90, 2056, 1500),
                                         ("bf16", 300, 32768, 1000), ("f16", 270, 1024, 900)])
def test_dz_takes_its_logits_as_the_losses_do(dtype, n, d, v):
    """p = exp(z - lse): what z loses over a long row of features would lower every p alike."""
    from dense_convolution_gb300 import head
    h, w, target = _positive(1, n, d, v, dtype, 4.0)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum")
    bias_h, bias_w, z = _signed_errors(h, w, target, op)
    # z: segments of at most 64 steps; the sums of dh and dw: v / 16 and n / 16
    # steps (twice where dz has two parts); the mean of the outputs' own roundings.
    for bias, k, count in ((bias_h, v, n * d), (bias_w, n, v * d)):
        assert abs(bias) < E * (64 * z + 64 + 2 * k / 16) + 4 * U[dtype] / math.sqrt(count), (bias, z)


@pytest.mark.parametrize("dtype,n,d,v,piece", [("f16", 1024, 4608, 100000, None), ("f16", 65536, 64, 19456, 19456),
                                               ("f16", 8192, 512, 65536, 65536), ("bf16", 1000, 4608, 200000, 200000)])
def test_long_sums_lose_less_than_their_rounding(dtype, n, d, v, piece):
    """dh sums over the vocabulary, dw over the tokens: no more than a fifth of the
    result's unit roundoff goes missing, however long they are."""
    from dense_convolution_gb300 import head
    h, w, target = _positive(2, n, d, v, dtype, 0.2)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum", piece=piece)
    bias_h, bias_w, z = _signed_errors(h, w, target, op, rounded=True)
    for bias, count in ((bias_h, n * d), (bias_w, v * d)):
        assert abs(bias) < U[dtype] / 5 + E * (64 * z + 64) + 4 * U[dtype] / math.sqrt(count), (bias, z)
