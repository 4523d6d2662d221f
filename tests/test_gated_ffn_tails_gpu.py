"""The feed-forward block's activations where they vanish, held relative to their own size, and where
their arguments overflow.

Hidden columns of g and of one, and weights that are unit vectors, make g and u = 1 exact, so that y = act(g) and,
from dy = 1, dx = (act'(g), act(g)); for one token u = g.  With u the unit roundoff of the type:
  act    fp32 and few tokens: exponentials are good to 2^-22, the normal distribution to 2^-20.7, and products
         round (2^-24 each): 2^-20 for silu, 2^-19 for gelu.  gelu_tanh's argument, up to 36 here, rounds five
         times: 36 5 2^-24 = 2^-16.5, with the rest 2^-16.  Long 16-bit ones: gelu_tanh's
         argument, up to 52 in powers of two, rounds five times for a fast exponential (2^-16); gelu's, up to 36, thrice
         (2^-17.3), and its tail's polynomial is off by 2^-15: 2^-14.5, beside the roundings of h and of y (u each).
  slope  near its zero (g = -0.75 for gelu) terms cancel: held to the sum of its two terms' magnitudes.
Values below the type's smallest normal one are held to half a step of the subnormal ones, twice.
"""
import math

import pytest

from .test_gated_ffn_gpu import U, _dt, _lib, _status  # noqa: F401

pytestmark = pytest.mark.gpu

STEP = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def _functions(act, g):
    """act(g), act'(g) and the sum of the magnitudes of its terms, in 64 bits."""
    import torch
    if act == "silu":
        s, q = torch.sigmoid(g), torch.sigmoid(-g)
        return g * s, s + g * s * q, s + (g * s * q).abs()
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        slope = g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * phi, phi + slope, phi + slope.abs()
    k, c = 2 * math.sqrt(2 / math.pi), 0.044715
    z = k * (g + c * g ** 3)
    s, q = torch.sigmoid(z), torch.sigmoid(-z)
    slope = g * s * q * k * (1 + 3 * c * g * g)
    return g * s, s + slope, s + slope.abs()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", [1, 600])
def test_tails_have_digits_of_their_own(act, dtype, t):
    import torch
    from dense_convolution_gb300 import head
    n = 600
    g = torch.linspace(-7, 3, n, device="cuda").to(_dt(dtype))
    one = lambda *shape: torch.ones(*shape, dtype=_dt(dtype), device="cuda")
    few, u = t == 1, U[dtype]
    rel = {"silu": 2.0 ** -20, "gelu": 2.0 ** -19, "gelu_tanh": 2.0 ** -16}[act] if few or dtype == "f32" else 2.0 ** -14.5
    a, slope, size = _functions(act, g.double())
    if few:
        # A token for each value would be slow: g lies in the weights, the values in the results of a single hidden column.
        for k in range(0, n, 7):
            op = head.GatedFeedForward(1, 1, 1, dtype, act)
            y = op(g[k].view(1, 1), one(1, 1), one(1, 1), one(1, 1)).double()
            off = (rel + u) * a[k].abs() + STEP[dtype]
            # (u = g here: h = act(g) g.)
            assert abs(float(y - a[k] * g[k].double())) <= float((off + u * a[k].abs()) * (1 + g[k].double().abs())), float(g[k])
        return
    # Two hidden columns: g is the first, u is the second, one.
    x = torch.stack([g, one(n)], 1)
    wg, wu, wd = one(1, 2), one(1, 2), one(2, 1)
    wg[0, 1] = wu[0, 0] = 0
    op = head.GatedFeedForward(n, 2, 1, dtype, act)
    y, saved = op(x, wg, wu, wd, save=True)
    off = (y[:, 0].double() - a).abs() / ((rel + 2 * u) * a.abs() + STEP[dtype])
    assert float(off.max()) <= 1, (float(off.max()), float(g[off.argmax()]))
    dy = torch.stack([one(n), torch.zeros_like(g)], 1)
    dx = op.backward(dy, x, wg, wu, wd, saved, need_dw=False)[0].double()
    # dx = [dg, du]: dg = act'(g), du = act(g).
    for got, want, scale in ((dx[:, 0], slope, size), (dx[:, 1], a, a.abs())):
        off = (got - want).abs() / ((2 * rel) * scale + 2 * u * want.abs() + STEP[dtype])
        assert float(off.max()) <= 1, (float(off.max()), float(g[off.argmax()]))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [2, 200])
def test_huge_pre_activations(act, dtype, t):
    """The slope of a finite pre-activation is 0 or 1 at the ends, whatever its powers overflow to."""
    import torch
    from dense_convolution_gb300 import head
    g = torch.tensor([1.0, -1.0, 1e12, -1e12, 3e13, -3e13, 1e20, -1e20, 1e30, -1e30, 3e38, -3e38], device="cuda").to(_dt(dtype))
    n = len(g)
    one = lambda *shape: torch.ones(*shape, dtype=_dt(dtype), device="cuda")
    x = one(t, 1)
    wg, wu, wd = g.view(n, 1).clone(), one(n, 1), one(1, n)
    wd *= 2.0 ** -4
    op = head.GatedFeedForward(t, 1, n, dtype, act)
    _, saved = op(x, wg, wu, wd, save=True)
    _, dwg, dwu, _ = op.backward(one(t, 1), x, wg, wu, wd, saved)
    slope = _functions(act, g.double())[1]
    want = t / 16 * torch.where(g.abs() > 2, (g > 0).double(), slope)
    assert torch.isfinite(dwg).all() and torch.isfinite(dwu[g < 1e38]).all()
    assert ((dwg[:, 0].double() - want).abs() <= (2 * U[dtype] + 2.0 ** -16) * want.abs() + 1e-30).all(), dwg[:, 0] - want
