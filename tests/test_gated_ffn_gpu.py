"""The gated feed-forward block against its definition in 64 bits, through the public
entry points.

With u the unit roundoff of the type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32; fp16 values
below 2^-14 round by up to 2^-25) and e = 2^-24, each result is held to the sum of
what its steps may be off by, terms and all taken in magnitude:
  sums of K 16-bit products   the tensor cores cut every 16 terms' sum toward zero (2 e
                each): c(K) = 2 e (K / 16 + 4) of the terms.
  fp32          three bf16 parts drop products below 4 e of each term; 24 cuts a segment
                (2 e each), a rounded addition for each 384 terms of each of six
                products: c(K) = e (60 + K / 32).
  act, act'     their arguments' error (|act'|, |act''| <= 1.2), and exponentials that are
                good to 6 2^-23 of 1: 2^-20 |g|, for act' 2^-19 (2 + |g|); fp32 an eighth.
  h, dg, du     one rounding to the type (none kept below fp32 for few tokens, which this
                still holds), fp16's dg and du on a scale where the largest |dy| is 16 at least.
  results       one rounding.
Summed in magnitude, roundings of h, dg and du are far over what they come to; so the
2-norms are held too: roundings are independent, of 0.43 u in the mean, two of them
(an operand's and the result's) make 0.6 u; 0.75 u leaves room for few terms.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _status():
    yield
    from dense_convolution_gb300 import capi
    assert capi.conv2d_device_status(0) == 0


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _inputs(seed, t, d, f, dtype, dy_scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda s, *shape: (torch.randn(*shape, generator=g, device="cuda") * s).to(_dt(dtype))
    return dict(x=randn(1.0, t, d), wg=randn(1.5 * d ** -0.5, f, d), wu=randn(d ** -0.5, f, d), wd=randn(f ** -0.5, d, f),
                residual=randn(1.0, t, d), dy=randn(dy_scale, t, d))


def _act(kind, g):
    import torch
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k, c = 2 * math.sqrt(2 / math.pi), 0.044715
    s = torch.sigmoid(k * (g + c * g ** 3))
    return g * s, s + g * s * (1 - s) * k * (1 + 3 * c * g * g)


def _reference(i, act, dtype):
    """{name: (value, bound)} in 64 bits."""
    x, wg, wu, wd, res, dy = (i[k].double() for k in ("x", "wg", "wu", "wd", "residual", "dy"))
    (t, d), f, u16 = x.shape, wg.shape[0], U[dtype]
    c = (lambda k: E * (60 + k / 32)) if dtype == "f32" else (lambda k: 2 * E * (k / 16 + 4))
    rough = 2.0 ** -20 if dtype != "f32" else 2.0 ** -23
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    xa, wga, wua, wda, dya = x.abs(), wg.abs(), wu.abs(), wd.abs(), dy.abs()
    g, u = x @ wg.T, x @ wu.T
    tg, tu = c(d) * (xa @ wga.T), c(d) * (xa @ wua.T)
    a, s = _act(act, g)
    ta, ts = 1.2 * tg + rough * g.abs(), 1.2 * tg + 2 * rough * (2 + g.abs())
    h = a * u
    th = ta * u.abs() + a.abs() * tu + ta * tu + (2 * E + u16) * h.abs() + tiny
    y = h @ wd.T
    out = {"y": (y + res, (th + c(f) * h.abs()) @ wda.T + (u16 + 2 * E) * (y + res).abs() + tiny)}
    dh = dy @ wd
    tdh = c(d) * (dya @ wda)
    tiny2 = tiny * float(dya.max()) / 16
    dg, du = dh * u * s, dh * a
    tdg = (dh.abs() + tdh) * ((u.abs() + tu) * (s.abs() + ts) - (u * s).abs()) + tdh * (u * s).abs() + (4 * E + u16) * dg.abs() + tiny2
    tdu = (dh.abs() + tdh) * ta + tdh * a.abs() + (4 * E + u16) * du.abs() + tiny2
    row = lambda v, b: (v, b + (u16 + 2 * E) * v.abs() + tiny)
    out["dx"] = row(dg @ wg + du @ wu, (tdg + c(2 * f) * dg.abs()) @ wga + (tdu + c(2 * f) * du.abs()) @ wua)
    out["dwg"] = row(dg.T @ x, (tdg + c(t) * dg.abs()).T @ xa)
    out["dwu"] = row(du.T @ x, (tdu + c(t) * du.abs()).T @ xa)
    out["dwd"] = row(dy.T @ h, dya.T @ (th + c(t) * h.abs()))
    return out


def _close(got, want, name, norm=None):
    import torch
    v, b = want
    g = got.double()
    assert torch.isfinite(g).all(), f"{name}: not finite"
    bad = (g - v).abs() > b
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {float(((g - v).abs() / b).max()):.2f} of the bound"
    if norm is not None:
        off = float((g - v).norm() / v.norm())
        assert off <= norm, f"{name}: off by {off:.3g} in the 2-norm, {norm:.3g} allowed"


def _run(op, i, **more):
    y, saved = op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"], save=True)
    dx, dwg, dwu, dwd = op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved, **more)
    return dict(y=y, dx=dx, dwg=dwg, dwu=dwu, dwd=dwd)


SIZES = [(1, 8, 8), (1, 1, 1), (2, 7, 5), (3, 64, 64), (5, 33, 129), (17, 128, 64), (128, 64, 128), (129, 200, 96),
         (300, 264, 1000), (777, 509, 137), (64, 2048, 300), (1000, 136, 520), (260, 1000, 72), (2100, 80, 328)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,d,f", SIZES)
def test_block(dtype, t, d, f):
    from dense_convolution_gb300 import head
    act = ("silu", "gelu", "gelu_tanh")[(t + d) % 3]
    i = _inputs(t * 7 + d, t, d, f, dtype)
    op = head.GatedFeedForward(t, d, f, dtype, act)
    got, want = _run(op, i), _reference(i, act, dtype)
    norm = 0.75 * U[dtype] if dtype != "f32" and t * d * f > 1e6 else 2e-6 if dtype == "f32" and t * d * f > 1e6 else None
    for k in want:
        _close(got[k], want[k], k, norm)
    # The same bits again, the same values without what is not wanted, and without a residual or what is saved.
    again = _run(op, i)
    assert all(again[k].equal(got[k]) for k in got)
    only = _run(op, i, need_dw=False)
    assert only["dx"].equal(got["dx"]) and only["dwg"] is None and only["dwd"] is None
    only = _run(op, i, need_dx=False)
    assert only["dx"] is None and all(only[k].equal(got[k]) for k in ("dwg", "dwu", "dwd"))
    assert op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"]).equal(got["y"])
    i["residual"].zero_()
    _close(op(i["x"], i["wg"], i["wu"], i["wd"]), _reference(i, act, dtype)["y"], "y alone")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", [2, 200])
def test_activations_far_from_zero(act, dtype, t):
    """Pre-activations from -60 to 60: neither overflow nor loss at the ends."""
    import torch
    from dense_convolution_gb300 import head
    d, f = 64, 160
    i = _inputs(5, t, d, f, dtype)
    i["x"][:] = 0
    i["x"][:, 0] = 1
    i["wg"][:, 0] = torch.linspace(-60, 60, f, device="cuda").to(_dt(dtype))
    op = head.GatedFeedForward(t, d, f, dtype, act)
    got, want = _run(op, i), _reference(i, act, dtype)
    for k in want:
        _close(got[k], want[k], k)


@pytest.mark.parametrize("t,d,f", [(130, 16384, 64), (20000, 64, 72), (140, 64, 40000)])
def test_sums_of_one_sign(t, d, f):
    """All terms positive, in fp16: what the tensor cores cut from long sums stays within the bounds."""
    from dense_convolution_gb300 import head
    i = _inputs(12, t, d, f, "f16")
    for k in ("x", "wg", "wu", "wd", "dy"):
        i[k].abs_()
    i["wg"] *= 2 / d ** 0.5                                # pre-activations near one
    i["wu"] *= 2 / d ** 0.5
    i["wd"] *= 2 / f ** 0.5
    i["dy"] *= min(1.0, 100 / t)
    op = head.GatedFeedForward(t, d, f, "f16", "silu")
    got, want = _run(op, i), _reference(i, "silu", "f16")
    for k in want:
        _close(got[k], want[k], k)


def _strided(v, stride, shift):
    """v's values in rows `stride` apart, `shift` elements into a buffer of NaN."""
    import torch
    rows, cols = v.shape
    buf = torch.full((shift + rows * stride + 8,), float("nan"), dtype=v.dtype, device="cuda")
    w = buf[shift:shift + rows * stride].as_strided((rows, cols), (stride, 1))
    w.copy_(v)
    return w, buf


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", [3, 150])
@pytest.mark.parametrize("d,f,xs,ys,x_shift,y_shift", [(64, 136, 72, 80, 0, 0), (64, 136, 67, 64, 3, 8), (50, 77, 50, 53, 1, 1),
                                                       (128, 64, 136, 131, 8, 5), (64, 64, 64, 72, 0, 4)])
def test_strides_alignment_and_buffers(dtype, t, d, f, xs, ys, x_shift, y_shift):
    import torch
    from dense_convolution_gb300 import head
    if dtype == "bf16" and y_shift % 8 and ys % 8 == 0:
        y_shift = 8                                        # rows that are read in place lie on 16 bytes
    if dtype == "f16" and y_shift % 8 and ys % 8 == 0:
        y_shift = 0
    i = _inputs(d + xs, t, d, f, dtype)
    want = _reference(i, "silu", dtype)
    i["x"], xbuf = _strided(i["x"], xs, x_shift)
    i["residual"], rbuf = _strided(i["residual"], ys, y_shift)
    i["dy"], _ = _strided(i["dy"], ys, y_shift)
    op = head.GatedFeedForward(t, d, f, dtype, "silu", x_stride=xs, y_stride=ys)
    # Workspaces full of NaN.
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (op.workspace_bytes, op.backward_workspace_bytes)]
    y, ybuf = _strided(torch.zeros(t, d, dtype=_dt(dtype), device="cuda"), ys, y_shift)
    _, saved = op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"], y=y, save=True, workspace=ws[0])
    got = dict(zip(("dx", "dwg", "dwu", "dwd"), op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved, workspace=ws[1])))
    got["y"] = y
    for k in want:
        _close(got[k], want[k], k)
    assert torch.isnan(ybuf).sum() == ybuf.numel() - t * d and torch.isnan(xbuf).sum() == xbuf.numel() - t * d
    # In place of the residual, and of x.
    op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"], y=i["residual"])
    assert i["residual"].equal(y) and torch.isnan(rbuf).sum() == rbuf.numel() - t * d
    if xs == ys and x_shift % 8 == y_shift % 8:
        op(i["x"], i["wg"], i["wu"], i["wd"], y=i["x"])
        _close(i["x"], (want["y"][0] - _inputs(d + xs, t, d, f, dtype)["residual"].double(), want["y"][1] + 2 * U[dtype]), "y in x's place")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", [4, 130])
def test_rows_that_are_not_finite_stay_alone(dtype, t):
    import torch
    from dense_convolution_gb300 import head
    d, f = 96, 200
    i = _inputs(3, t, d, f, dtype)
    op = head.GatedFeedForward(t, d, f, dtype, "gelu")
    clean = _run(op, i)
    i["x"][1, 5], i["x"][3, 0] = float("nan"), float("inf")
    y = op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"])
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[[1, 3]] = False
    assert y[keep].equal(clean["y"][keep]) and torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()
    y, saved = op(i["x"], i["wg"], i["wu"], i["wd"], save=True)
    dx = op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved, need_dw=False)[0]
    assert dx[keep].equal(clean["dx"][keep]) and torch.isnan(dx[1]).all()


@pytest.mark.parametrize("scale", [60000.0 / 6, 1e-6])
def test_fp16_gradients_of_any_size(scale):
    """The scale of dg and du follows dy: neither lost nor infinite on the way."""
    from dense_convolution_gb300 import head
    t, d, f = 300, 128, 256
    i = _inputs(8, t, d, f, "f16", dy_scale=scale)
    op = head.GatedFeedForward(t, d, f, "f16", "silu")
    if scale > 1:                                          # the weights' gradients stay inside fp16
        i["x"] /= 256
        i["wu"] /= 64
    got, want = _run(op, i), _reference(i, "silu", "f16")
    for k in ("dx", "dwg", "dwu", "dwd"):
        _close(got[k], want[k], k)
    i["dy"].zero_()
    got = _run(op, i)
    assert not any(got[k].any() for k in ("dx", "dwg", "dwu", "dwd"))


@pytest.mark.parametrize("t,d,f", [(40, 24, 50), (3, 16, 40), (150, 130, 70)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(t, d, f, act):
    import torch
    from dense_convolution_gb300 import head
    i = _inputs(11, t, d, f, "f32")
    op = head.GatedFeedForward(t, d, f, "f32", act)
    got = _run(op, i)
    v = {k: x.double() for k, x in i.items()}

    def loss(v):
        a, _ = _act(act, v["x"] @ v["wg"].T)
        return float((((a * (v["x"] @ v["wu"].T)) @ v["wd"].T) * v["dy"]).sum())

    g = torch.Generator(device="cuda").manual_seed(1)
    for k, grad in (("x", "dx"), ("wg", "dwg"), ("wu", "dwu"), ("wd", "dwd")):
        way = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
        way /= way.norm()
        h = 1e-4
        diff = (loss({**v, k: v[k] + h * way}) - loss({**v, k: v[k] - h * way})) / (2 * h)
        # The third derivative's share is h^2 times the gradient's size or so.
        assert abs(diff - float((got[grad].double() * way).sum())) <= 1e-6 * (1 + float(got[grad].double().norm())), k


@pytest.mark.parametrize("t", [4, 200])
def test_other_stream_and_capture(t):
    import torch
    from dense_convolution_gb300 import head
    d, f = 128, 320
    i = _inputs(2, t, d, f, "f16")
    op = head.GatedFeedForward(t, d, f, "f16", "silu")
    want = _run(op, i)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, saved = op(i["x"], i["wg"], i["wu"], i["wd"], residual=i["residual"], save=True, stream=side)
    grads = op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved, stream=side)
    side.synchronize()
    assert y.equal(want["y"]) and all(a.equal(want[k]) for a, k in zip(grads, ("dx", "dwg", "dwu", "dwd")))
    # Two graphs of one workspace, replayed in turn with other inputs.
    ws = torch.empty(max(op.workspace_bytes, op.backward_workspace_bytes), dtype=torch.uint8, device="cuda")
    j = _inputs(3, t, d, f, "f16")
    graphs, outs = [], []
    for inputs in (i, {k: v.clone() for k, v in i.items()}):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, saved = op(inputs["x"], inputs["wg"], inputs["wu"], inputs["wd"], residual=inputs["residual"], save=True, workspace=ws)
            outs.append((inputs, y, op.backward(inputs["dy"], inputs["x"], inputs["wg"], inputs["wu"], inputs["wd"], saved, workspace=ws)))
        graphs.append(graph)
    for k, v in j.items():
        outs[1][0][k].copy_(v)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for w, (_, y, grads) in zip((want, _run(op, j)), outs):
        assert y.equal(w["y"]) and all(a.equal(w[k]) for a, k in zip(grads, ("dx", "dwg", "dwu", "dwd")))


def test_beyond_32_bit_offsets():
    """What is saved passes 2^31 elements: the last rows are those of a small call."""
    import torch
    from dense_convolution_gb300 import head
    t, d, f, few = 280000, 64, 4096, 300
    g = torch.Generator(device="cuda").manual_seed(4)
    i = _inputs(4, few, d, f, "bf16")
    x = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    dy = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    x[-few:], dy[-few:] = i["x"], i["dy"]
    op, small = head.GatedFeedForward(t, d, f, "bf16"), head.GatedFeedForward(few, d, f, "bf16")
    y, saved = op(x, i["wg"], i["wu"], i["wd"], save=True)
    want = _reference({**i, "residual": torch.zeros_like(i["x"])}, "silu", "bf16")
    _close(y[-few:], want["y"], "y")
    dx, dwg, dwu, dwd = op.backward(dy, x, i["wg"], i["wu"], i["wd"], saved)
    _close(dx[-few:], want["dx"], "dx")
    assert not dx[:-few].any()
    for k, v in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        _close(v, want[k], k, 0.75 * U["bf16"])


@pytest.mark.parametrize("dtype,t,d,f", [("bf16", 300, 264, 520), ("f32", 200, 72, 130)])
def test_each_gradient_alone_has_the_same_bits(dtype, t, d, f):
    import itertools

    import torch
    from dense_convolution_gb300 import head, head_capi
    i = _inputs(9, t, d, f, dtype)
    op = head.GatedFeedForward(t, d, f, dtype)
    _, saved = op(i["x"], i["wg"], i["wu"], i["wd"], save=True)
    want = op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved)
    ws = torch.empty(op.backward_workspace_bytes, dtype=torch.uint8, device="cuda")
    for wanted in itertools.product((False, True), repeat=4):
        out = [torch.full_like(v, float("nan")) for v in want]
        head_capi.gated_ffn_bwd(op.desc, i["dy"].data_ptr(), i["x"].data_ptr(), i["wg"].data_ptr(), i["wu"].data_ptr(),
                                i["wd"].data_ptr(), saved.data_ptr(), *(o.data_ptr() if w else 0 for o, w in zip(out, wanted)),
                                ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        for o, v, w in zip(out, want, wanted):
            assert o.equal(v) if w else torch.isnan(o).all(), wanted


def test_threads_with_shapes_of_their_own():
    """Calls of one kernel from several threads: what one shape needs of it (its shared memory) takes nothing from another's."""
    import threading

    import torch
    from dense_convolution_gb300 import head
    start, errors = threading.Barrier(4), []

    def loop(t, d, f, dtype):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                i = _inputs(t, t, d, f, dtype)
                op = head.GatedFeedForward(t, d, f, dtype)
                want = _run(op, i)
                stream.synchronize()
                start.wait()
                for _ in range(200):
                    got = _run(op, i)
                stream.synchronize()
                assert all(got[k].equal(want[k]) for k in want)
        except Exception as e:
            errors.append(repr(e))
            start.abort()

    threads = [threading.Thread(target=loop, args=a) for a in ((3, 4096, 64, "bf16"), (3, 64, 96, "bf16"), (300, 512, 512, "bf16"),
                                                               (140, 33, 47, "bf16"))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_no_tokens():
    import torch
    from dense_convolution_gb300 import head
    i = _inputs(1, 1, 8, 24, "bf16")
    op = head.GatedFeedForward(0, 8, 24, "bf16")
    none = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    y, saved = op(none, i["wg"], i["wu"], i["wd"], save=True)
    dx, *dw = op.backward(none, none, i["wg"], i["wu"], i["wd"], saved)
    assert y.shape == dx.shape == (0, 8) and not any(w.any() for w in dw)


def test_wrong_tensors_are_refused():
    import torch
    from dense_convolution_gb300 import head
    t, d, f = 20, 16, 40
    i = _inputs(1, t, d, f, "bf16")
    op = head.GatedFeedForward(t, d, f, "bf16")
    y, saved = op(i["x"], i["wg"], i["wu"], i["wd"], save=True)
    base = {k: i[k] for k in ("x", "wg", "wu", "wd")}
    for k, v in (("x", i["x"][:-1]), ("x", i["x"].half()), ("x", i["x"].cpu()), ("wg", i["wd"]), ("wu", i["wu"].float()),
                 ("wd", i["wg"]), ("wd", i["wg"].T), ("residual", i["x"][1:]), ("y", torch.empty(t, d + 8, dtype=torch.bfloat16, device="cuda")[:, :d]),
                 ("workspace", torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            op(**{**base, k: v})
    base = {**base, "dy": i["dy"], "saved": saved}
    for k, v in (("dy", i["dy"].float()), ("saved", saved[:-1]), ("saved", saved.half()), ("wd", i["wg"])):
        with pytest.raises(ValueError):
            op.backward(**{**base, k: v})
    from dense_convolution_gb300 import capi
    with pytest.raises(capi.Conv2dError):
        op.backward(**base, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("t,d,f,dtype", [(600, 512, 900, "bf16"), (100, 256, 700, "f16"), (300, 320, 500, "f32")])
@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_that_runs_out_is_reported(t, d, f, dtype, backward):
    import torch
    from dense_convolution_gb300 import capi, head
    i = _inputs(6, t, d, f, dtype)
    op = head.GatedFeedForward(t, d, f, dtype)
    y, saved = op(i["x"], i["wg"], i["wu"], i["wd"], save=True)
    call = (lambda: op.backward(i["dy"], i["x"], i["wg"], i["wu"], i["wd"], saved)) if backward else (
        lambda: op(i["x"], i["wg"], i["wu"], i["wd"], save=True)[:1])     # (what is saved ends in rows that nobody reads)
    want = [v.clone() for v in call()]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    try:
        capi.conv2d_set_wait_limit(1, stream)
        call()
        torch.cuda.synchronize()
        assert capi.conv2d_device_status(stream) != 0
    finally:
        capi.conv2d_set_wait_limit(0, stream)
    assert all(a.equal(b) for a, b in zip(want, call()))
