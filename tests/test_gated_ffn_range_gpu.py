"""fp16 gradients of the feed-forward block whose dg and du are far from dy: held as fp16 numbers on
a scale of their own, none is infinite or without digits where the results are fp16 numbers.

Bounds are those of test_gated_ffn_gpu, with one term of its own: the largest |dg| or |du| is
held at 2^10 at least, so that what is held in subnormal numbers is off by up to 2^-25, 2^-35 of the largest.
A row's own digits: dg, du and the result round by 0.43 u in the mean, together 0.6 u in the
2-norm.  In a row 2^-20 of the largest, whose dg are 2^-3 of their own largest in the mean, 2^-25 3^(-1/2) on 2^-13 adds 0.3 u:
0.67 u.  A row's 2-norm over some 256 results, the large ones counting most, strays by a fourteenth, and the worst of
300 rows by three times that: 0.81 u, and 0.85 u is allowed.
"""
import pytest

from .test_gated_ffn_gpu import U, _act, _close, _inputs, _lib, _reference, _run, _status  # noqa: F401

pytestmark = pytest.mark.gpu


def _bounds(i, act):
    """test_gated_ffn_gpu's, with what the scale of dg and du costs at most."""
    want = _reference(i, act, "f16")
    x, wg, wu, wd, dy = (i[k].double() for k in ("x", "wg", "wu", "wd", "dy"))
    a, s = _act(act, x @ wg.T)
    dh = dy @ wd
    dg, du = dh * (x @ wu.T) * s, dh * a
    top = max(float(dg.abs().max()), float(du.abs().max()))
    tiny = 2.0 ** -35 * top
    rows = wg.abs().sum(0) + wu.abs().sum(0)
    cols = x.abs().sum(0)
    for k, more in (("dx", rows), ("dwg", cols), ("dwu", cols)):
        want[k] = (want[k][0], want[k][1] + tiny * more)
    return want, top


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,d,f", [(512, 4096, 128), (100, 2900, 70), (700, 2000, 600), (3, 2048, 64)])
def test_large_gradients_from_a_small_dy(t, d, f, act):
    """|dg| is thousands of times the largest |dy|: all true values are fp16 numbers."""
    from dense_convolution_gb300 import head
    i = _inputs(t + f, t, d, f, "f16")
    i["wg"] *= 2 / 3                                       # deviation hidden^(-1/2)
    i["wu"] *= d ** 0.5
    i["wd"] *= 4 * f ** 0.5
    i["dy"] *= 1e-3
    want, top = _bounds(i, act)
    assert 4096 * float(i["dy"].abs().max()) < top < 65504
    got = _run(head.GatedFeedForward(t, d, f, "f16", act), i)
    for k in want:
        assert float(want[k][0].abs().max()) < 65000
        _close(got[k], want[k], k, 0.75 * U["f16"] if t * d * f > 1e6 and k != "y" else None)


def test_each_large_gradient_alone_has_the_same_bits():
    import torch
    from dense_convolution_gb300 import head
    t, d, f = 300, 1024, 200
    i = _inputs(2, t, d, f, "f16")
    i["wu"] *= d ** 0.5
    i["wd"] *= 4 * f ** 0.5
    i["dy"] *= 1e-3
    op = head.GatedFeedForward(t, d, f, "f16")
    got = _run(op, i)
    only = _run(op, i, need_dw=False)
    assert only["dx"].equal(got["dx"])
    only = _run(op, i, need_dx=False)
    assert all(only[k].equal(got[k]) for k in ("dwg", "dwu", "dwd"))
    # Captured, and replayed with gradients that want another scale than the first ones.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _run(op, i)
    small = i["dy"].clone()
    for factor in (1.0, 0.01, 16.0):
        i["dy"].copy_(small * factor)
        graph.replay()
        now = _run(op, i)
        assert all(held[k].equal(now[k]) and torch.isfinite(now[k]).all() for k in now), factor


@pytest.mark.parametrize("t,d,f", [(300, 256, 512), (90, 300, 200)])
@pytest.mark.parametrize("wd_scale,gap", [(2.0 ** -6, 2.0 ** 14), (2.0 ** -3, 2.0 ** 20), (1.0, 2.0 ** 20), (2.0 ** 6, 2.0 ** 20)])
def test_rows_of_other_sizes_keep_their_digits(t, d, f, wd_scale, gap):
    """A few rows' dy is `gap` times the others': each row of dx is held to its own size."""
    from dense_convolution_gb300 import head
    i = _inputs(17, t, d, f, "f16", dy_scale=2.0 ** -11 / wd_scale)
    i["wd"] *= wd_scale
    i["dy"][5:8] *= gap
    want, _ = _bounds(i, "silu")
    got = _run(head.GatedFeedForward(t, d, f, "f16", "silu"), i, need_dw=False)
    v = want["dx"][0]
    assert 2.0 ** -12 < float(v[20:].square().mean().sqrt()) and float(v.abs().max()) < 65000
    off = ((got["dx"].double() - v).norm(dim=1) / v.norm(dim=1)).max()
    assert float(off) <= 0.85 * U["f16"], float(off) / U["f16"]


@pytest.mark.parametrize("t", [40, 300])
def test_rows_that_are_not_finite_leave_the_others_their_digits(t):
    """The scale goes by the finite values: du of some 2^-17 keeps its digits beside a row of NaN."""
    import torch
    from dense_convolution_gb300 import head
    d, f = 256, 512
    i = _inputs(23, t, d, f, "f16", dy_scale=2.0 ** -17)
    i["wu"] *= 2.0 ** 8
    want, _ = _bounds(i, "silu")
    i["dy"][5], i["dy"][7, 3], i["x"][11, 2] = float("nan"), float("inf"), float("inf")
    got = _run(head.GatedFeedForward(t, d, f, "f16", "silu"), i, need_dw=False)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[[5, 7, 11]] = False
    v = want["dx"][0][keep]
    off = ((got["dx"][keep].double() - v).norm(dim=1) / v.norm(dim=1)).max()
    assert float(off) <= 0.85 * U["f16"], float(off) / U["f16"]
    assert not torch.isfinite(got["dx"][~keep]).all(dim=1).any()
