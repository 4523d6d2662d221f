"""The training-head operators against their definitions in 64 bits, through the
public entry points.

Tolerances follow from the arithmetic.  With u the unit roundoff of the output
type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32; fp16 values below 2^-14 round to
multiples of 2^-24, by up to 2^-25 whatever their size) and e = 2^-24 that of
fp32:
  layer norm    one rounding to the output, and fp32 sums whose trees and chains
                are below 64 additions deep: u |y| + 64 e (sum of the terms'
                magnitudes).
  dropout       the product and the addition round in fp32, then once: the mask
                is exact.
  linear_ce     a product of 16-bit values is exact in fp32; an accumulation
                step on the tensor cores rounds toward zero (2 e each): 16 steps
                per 256-wide segment and one addition per segment.  dz is rounded
                to the operand type (u16) before dh and dw, whose sums run for
                K / 16 steps.  fp32 operands: three bf16 parts, whose dropped
                products are below 4 e of each term.
"""
import math

import numpy as np
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


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def _strided(t, stride, shift=0):
    """t's values in rows `stride` apart, `shift` elements into a buffer of NaN."""
    import torch
    rows, cols = t.shape
    buf = torch.full((shift + rows * stride + 8,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[shift:shift + rows * stride].as_strided((rows, cols), (stride, 1))
    v.copy_(t)
    return v, buf


def _close(got, want, tol, what):
    import torch
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = ((g - want).abs() > tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(((g - want).abs() / tol).max()):.2f} of the tolerance"


# ------------------------------------------------------------------ layer norm
def _norm_reference(x, gamma, beta, eps, dy=None, stats=None):
    """y, mean, rstd (, dx, dgamma, dbeta) in 64 bits, and the magnitudes the tolerances use."""
    x, g, b = x.double(), gamma.double(), beta.double()
    if stats is None:
        mean = x.mean(1)
        rstd = ((x - mean[:, None]).square().mean(1) + eps).rsqrt()
    else:
        mean, rstd = stats[0].double(), stats[1].double()
    z = (x - mean[:, None]) * rstd[:, None]
    big = (x.abs() + mean.abs()[:, None]) * rstd[:, None]
    out = {"y": z * g + b, "mean": mean, "rstd": rstd, "y_size": big * g.abs() + b.abs(),
           "mean_size": x.abs().mean(1), "rstd_size": rstd * (1 + (big * big).mean(1).clamp_max(1e6))}
    if dy is not None:
        d = dy.double()
        a = d * g
        out["dx"] = rstd[:, None] * (a - a.mean(1, keepdim=True) - z * (a * z).mean(1, keepdim=True))
        out["dx_size"] = rstd[:, None] * (a.abs() + a.abs().mean(1, keepdim=True)
                                          + big * (a.abs() * big).mean(1, keepdim=True))
        out["dgamma"], out["dgamma_size"] = (d * z).sum(0), (d.abs() * big).sum(0)
        out["dbeta"], out["dbeta_size"] = d.sum(0), d.abs().sum(0)
    return out


def _check_norm(op, x, rows_of, gamma, beta, dy, dtype, param, eps=1e-5):
    y, mean, rstd = op(x, gamma, beta, stats=True)
    r = _norm_reference(rows_of(x), gamma, beta, eps, dy, None)
    _close(y, r["y"], U[dtype] * r["y"].abs() + 64 * E * r["y_size"], "y")
    _close(mean, r["mean"], 64 * E * r["mean_size"] + 1e-30, "mean")
    _close(rstd, r["rstd"], 64 * E * r["rstd_size"], "rstd")
    dx, dgamma, dbeta = op.backward(dy, x, gamma, mean, rstd)
    r = _norm_reference(rows_of(x), gamma, beta, eps, dy, (mean, rstd))
    _close(rows_of(dx), r["dx"], U[dtype] * r["dx"].abs() + 64 * E * r["dx_size"], "dx")
    _close(dgamma, r["dgamma"], U[param] * r["dgamma"].abs() + 64 * E * r["dgamma_size"] + 1e-30, "dgamma")
    _close(dbeta, r["dbeta"], U[param] * r["dbeta"].abs() + 64 * E * r["dbeta_size"] + 1e-30, "dbeta")
    # The same bits again, and the same values without the outputs that are not
    # wanted (where dx lies decides whether vectors move, so the order of sums may differ).
    again = op.backward(dy, x, gamma, mean, rstd)
    only_dx = op.backward(dy, x, gamma, mean, rstd, need_params=False)
    only_params = op.backward(dy, x, gamma, mean, rstd, need_dx=False)
    assert again[0].equal(dx) and again[1].equal(dgamma) and again[2].equal(dbeta)
    assert only_dx[0].equal(dx) and only_dx[1] is None and only_params[0] is None
    _close(only_params[1], r["dgamma"], U[param] * r["dgamma"].abs() + 64 * E * r["dgamma_size"] + 1e-30, "dgamma alone")
    _close(only_params[2], r["dbeta"], U[param] * r["dbeta"].abs() + 64 * E * r["dbeta_size"] + 1e-30, "dbeta alone")
    return y, mean, rstd, dx


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 64), (1000, 32), (257, 100), (1, 4096), (33, 1000),
                                       (700, 771), (1300, 2048), (311, 4097), (650, 8192), (9, 8185), (3, 20001),
                                       (2, 65536), (1, 300000), (40, 9000), (700, 3000), (1300, 2040), (5000, 512), (2600, 1024)])
def test_layernorm_rows(dtype, rows, cols):
    from dense_convolution_gb300 import head
    g = _gen(rows * 100003 + cols)
    x = (_randn(g, rows, cols) * 1.5 + 0.4).to(_dt(dtype))
    dy = _randn(g, rows, cols).to(_dt(dtype))
    for param in {dtype, "f32"}:
        gamma, beta = (1 + 0.1 * _randn(g, cols)).to(_dt(param)), _randn(g, cols).to(_dt(param))
        op = head.LayerNorm(rows, cols, dtype, param)
        _check_norm(op, x, lambda t: t, gamma, beta, dy, dtype, param)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,xs,ys,x_shift,y_shift", [
    (60, 48, 56, 48, 0, 0), (37, 33, 40, 33, 0, 0), (29, 100, 103, 103, 3, 3), (29, 100, 103, 101, 3, 0),
    (64, 512, 513, 513, 0, 0), (17, 2048, 2051, 2053, 1, 5), (5, 9001, 9003, 9003, 2, 2), (700, 1024, 1040, 1032, 0, 0)])
def test_layernorm_strides_and_alignment(dtype, rows, cols, xs, ys, x_shift, y_shift):
    import torch
    from dense_convolution_gb300 import head
    g = _gen(cols + xs)
    x, xbuf = _strided((_randn(g, rows, cols) - 0.3).to(_dt(dtype)), xs, x_shift)
    dy, _ = _strided(_randn(g, rows, cols).to(_dt(dtype)), ys, y_shift)
    gamma = (1 + 0.1 * _randn(g, cols + 1)).to(_dt(dtype))[1:]          # off the 16-byte boundary
    beta = _randn(g, cols + 1).to(_dt(dtype))[1:]
    op = head.LayerNorm(rows, cols, dtype, dtype, x_stride=xs, y_stride=ys)
    y, mean, rstd, dx = _check_norm(op, x, lambda t: t, gamma, beta, dy, dtype, dtype)
    # Into given buffers: what lies between the rows stays.
    out, buf = _strided(torch.zeros_like(y), ys, y_shift)
    op(x, gamma, beta, y=out)
    r = _norm_reference(x, gamma, beta, 1e-5)
    _close(out, r["y"], U[dtype] * r["y"].abs() + 64 * E * r["y_size"], "y in place of a buffer")
    assert torch.isnan(buf).sum() == buf.numel() - rows * cols
    if xs == ys and x_shift == y_shift:                                   # in place
        assert op(x, gamma, beta, y=x).equal(out)
        assert torch.isnan(xbuf).sum() == xbuf.numel() - rows * cols


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("images,cols,pixels", [(1, 1, 1), (2, 5, 3), (3, 64, 49), (2, 512, 784), (2, 96, 196),
                                                (5, 72, 40), (1, 1024, 64), (2, 1000, 25), (3, 130, 36), (1, 2048, 16),
                                                (2, 4000, 9), (4, 300, 8), (40, 64, 400), (1, 16384, 3)])
def test_layernorm_planes(dtype, images, cols, pixels):
    from dense_convolution_gb300 import head
    g = _gen(cols * 7 + pixels)
    rows = images * pixels
    x = (_randn(g, images, cols, pixels) + 0.5 * _randn(g, 1, cols, 1)).to(_dt(dtype))
    dy = _randn(g, rows, cols).to(_dt(dtype))
    gamma, beta = 1 + 0.1 * _randn(g, cols), _randn(g, cols)
    op = head.LayerNorm(rows, cols, dtype, "f32", pixels=pixels)
    _check_norm(op, x, lambda t: t.reshape(images, cols, pixels).transpose(1, 2).reshape(rows, cols), gamma, beta, dy,
                dtype, "f32")


def test_layernorm_planes_into_strided_rows_and_unaligned_planes():
    import torch
    from dense_convolution_gb300 import capi, head, head_capi
    g = _gen(5)
    images, cols, pixels = 2, 64, 48
    rows = images * pixels
    gamma, beta = 1 + 0.1 * _randn(g, cols), _randn(g, cols)
    for shift in (0, 4, 1):
        flat = torch.randn(images * cols * pixels + 8, generator=g, device="cuda").to(torch.bfloat16)
        x = flat[shift:shift + images * cols * pixels].view(images, cols, pixels)
        dy, _ = _strided(_randn(g, rows, cols).to(torch.bfloat16), 67, 1)
        op = head.LayerNorm(rows, cols, "bf16", "f32", pixels=pixels, y_stride=67)
        _check_norm(op, x, lambda t: t.transpose(1, 2).reshape(rows, cols), gamma, beta, dy, "bf16", "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layernorm_constant_rows_and_no_parameters(dtype):
    import torch
    from dense_convolution_gb300 import head
    rows, cols = 9, 264
    x = torch.full((rows, cols), 3.0, device="cuda", dtype=_dt(dtype))
    x[4] = torch.arange(cols, device="cuda") % 2                          # one row that varies
    op = head.LayerNorm(rows, cols, dtype)
    y, mean, rstd = op(x, stats=True)
    assert (y[0] == 0).all() and mean[0] == 3.0
    assert abs(float(rstd[0]) - 1 / math.sqrt(1e-5)) < 1e-3
    assert abs(float(y[4, 1]) - 1) < 1e-2 and abs(float(y[4, 0]) + 1) < 1e-2
    dx, dgamma, dbeta = op.backward(torch.ones_like(x), x, None, mean, rstd)
    assert (dx[0] == 0).all() and (dbeta == rows).all()


def test_layernorm_nan_and_infinity_stay_in_their_row():
    import torch
    from dense_convolution_gb300 import head
    for rows, cols in ((6, 100), (6, 4096), (400, 2048)):
        x = _randn(_gen(3), rows, cols).to(torch.bfloat16)
        x[1, 5], x[3, 7] = float("nan"), float("inf")
        op = head.LayerNorm(rows, cols, "bf16")
        y, mean, rstd = op(x, stats=True)
        keep = [i for i in range(rows) if i not in (1, 3)]
        assert torch.isnan(y[1]).all() and torch.isnan(y[3]).any()
        assert torch.isfinite(y[keep].float()).all()
        dx, _, _ = op.backward(torch.ones_like(x), x, None, mean, rstd)
        assert torch.isfinite(dx[keep].float()).all()


def test_layernorm_beyond_32_bit_offsets():
    """Rows whose elements lie past 2^32 from the first, forward and backward."""
    import torch
    from dense_convolution_gb300 import head
    rows, cols = 66000, 65536
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.float16)
    g = _gen(9)
    tail = (_randn(g, 3, cols) + 0.2).half()
    x[-3:] = tail
    x[:3] = tail.flip(0)
    op = head.LayerNorm(rows, cols, "f16", "f32")
    y, mean, rstd = op(x, stats=True)
    one = torch.ones(cols, device="cuda")
    r = _norm_reference(tail, one, 0 * one, 1e-5)
    for got, want in ((y[-3:], r["y"]), (y[:3].flip(0), r["y"])):
        _close(got, want, U["f16"] * want.abs() + 64 * E * r["y_size"], "y")
    assert not y[3:-3].any()
    dx, _, _ = op.backward(x, x, None, mean, rstd, need_params=False)
    r = _norm_reference(tail, one, 0 * one, 1e-5, tail, (mean[-3:], rstd[-3:]))
    _close(dx[-3:], r["dx"], U["f16"] * r["dx"].abs() + 64 * E * r["dx_size"], "dx")


def test_layernorm_no_rows():
    import torch
    from dense_convolution_gb300 import head
    op = head.LayerNorm(0, 16, "f16", "f32")
    x = torch.empty(0, 16, device="cuda", dtype=torch.float16)
    y, mean, rstd = op(x, stats=True)
    assert y.shape == (0, 16)
    dx, dgamma, dbeta = op.backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 16) and (dgamma == 0).all() and (dbeta == 0).all()


@pytest.mark.parametrize("rows,cols,pixels", [(13, 120, None), (1300, 512, None), (3, 9000, None), (98, 40, 49)])
def test_layernorm_gradient_against_differences(rows, cols, pixels):
    """<dx, d> = the derivative of <dy, y> along d, by central differences: the
    truncation is of order step^2 and the fp32 rounding of order e / step."""
    import torch
    from dense_convolution_gb300 import head
    g = _gen(rows)
    shape = (rows // pixels, cols, pixels) if pixels else (rows, cols)
    x, d, dy = _randn(g, *shape), _randn(g, *shape), _randn(g, rows, cols)
    gamma, beta = 1 + 0.1 * _randn(g, cols), _randn(g, cols)
    op = head.LayerNorm(rows, cols, "f32", pixels=pixels)
    _, mean, rstd = op(x, gamma, beta, stats=True)
    dx, dgamma, dbeta = op.backward(dy, x, gamma, mean, rstd)
    h = 1e-2
    val = lambda x, gm, b: (dy.double() * op(x, gm, b).double()).sum()
    # The sums are over rows * cols terms of size one: scale the tolerance by their spread.
    tol = 1e-3 * math.sqrt(rows * cols)
    assert abs(float((val(x + h * d, gamma, beta) - val(x - h * d, gamma, beta)) / (2 * h) - (dx.double() * d).sum())) < tol
    e = _randn(g, cols)
    assert abs(float((val(x, gamma + h * e, beta) - val(x, gamma - h * e, beta)) / (2 * h) - (dgamma.double() * e).sum())) < tol
    assert abs(float((val(x, gamma, beta + h * e) - val(x, gamma, beta - h * e)) / (2 * h) - (dbeta.double() * e).sum())) < tol


# ------------------------------------------------------------------ dropout
def _philox(seed, offset, blocks, stream):
    """Philox4x32-10 in plain Python integers (numpy uint64), words of each block."""
    low = np.uint64(0xFFFFFFFF)
    i = np.arange(blocks, dtype=np.uint64)
    c = [i & low, i >> np.uint64(32), np.full(blocks, offset & 0xFFFFFFFF, np.uint64),
         np.full(blocks, (offset >> 32) | (stream << 31), np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1)


def _keep(seed, offset, n, p):
    """The mask from its definition (include/head.h)."""
    blocks = -(-n // 8)
    half = []
    for s in (0, 1):
        w = _philox(seed, offset, blocks, s)
        half.append(np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:n])
    return ((half[0] << np.uint64(16)) | half[1]) >= np.uint64(round(p * 2 ** 32))


def test_philox_reference_against_the_published_vectors():
    """The known answers of Philox4x32-10 for an all-zero and an all-one input."""
    assert [int(v) for v in _philox(0, 0, 1, 0)[0]] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,xs,rs,ys,shift,p", [
    (1, 1, 1, 1, 1, 0, 0.5), (3, 5, 5, 5, 5, 0, 0.3), (7, 1001, 1001, 1001, 1001, 0, 0.5), (40, 64, 64, 64, 64, 0, 0.1),
    (40, 64, 72, 64, 80, 0, 0.1), (33, 100, 101, 102, 103, 1, 0.25), (500, 2048, 2048, 2048, 2048, 0, 0.1),
    (9, 3, 3, 3, 3, 1, 0.7), (12, 40, 40, 40, 40, 0, 0.0), (12, 40, 40, 40, 40, 0, 1.0)])
def test_dropout(dtype, rows, cols, xs, rs, ys, shift, p):
    import torch
    from dense_convolution_gb300 import head
    g = _gen(rows + cols)
    seed, offset = 0xDEADBEEF12345678, (5 << 32) + 77
    x, _ = _strided(_randn(g, rows, cols).to(_dt(dtype)), xs, shift)
    res, _ = _strided(_randn(g, rows, cols).to(_dt(dtype)), rs, shift)
    dy, _ = _strided(_randn(g, rows, cols).to(_dt(dtype)), ys, shift)
    op = head.Dropout(rows, cols, dtype, p, x_stride=xs, residual_stride=rs, y_stride=ys)
    keep = torch.from_numpy(_keep(seed, offset, rows * cols, p).reshape(rows, cols)).cuda()
    scale = 1 / (1 - p) if p < 1 else 0.0
    want = torch.where(keep, x.double() * scale, 0.0)
    tol = (U[dtype] + 2 * E) * want.abs()
    y = op(x, seed, offset)
    assert ((y == 0) | keep).all()
    _close(y, want, tol, "y")
    total = want + res.double()
    _close(op(x, seed, offset, residual=res), total, U[dtype] * total.abs() + 3 * E * (want.abs() + res.double().abs()),
           "y with residual")
    back = torch.where(keep, dy.double() * scale, 0.0)
    dx = op.backward(dy, seed, offset)
    _close(dx, back, (U[dtype] + 2 * E) * back.abs(), "dx")
    out, buf = _strided(torch.zeros(rows, cols, dtype=_dt(dtype), device="cuda"), ys, shift)
    assert op(x, seed, offset, y=out).equal(y)
    assert torch.isnan(buf).sum() == buf.numel() - rows * cols            # between the rows nothing is written


def test_dropout_ties_take_the_low_half():
    """A threshold whose high half is met by many elements: only the second
    stream's bits separate them."""
    import torch
    from dense_convolution_gb300 import head
    rows, cols, seed = 4096, 1024, 99
    x = torch.ones(rows, cols, device="cuda")
    p = (0x8000 * 65536 + 0x7FFF) / 2 ** 32
    y = head.Dropout(rows, cols, "f32", p)(x, seed, 3)
    keep = torch.from_numpy(_keep(seed, 3, rows * cols, p).reshape(rows, cols)).cuda()
    high = _philox(seed, 3, rows * cols // 8, 0)
    ties = int(((high & np.uint64(0xFFFF)) == 0x8000).sum() + ((high >> np.uint64(16)) == 0x8000).sum())
    assert ties > 20                                                       # about 64 expected
    assert ((y != 0) == keep).all()


def test_dropout_rate_seeds_and_dropped_nan():
    import torch
    from dense_convolution_gb300 import head
    n, p = 1 << 20, 0.3
    x = torch.ones(1, n, device="cuda", dtype=torch.float16)
    op = head.Dropout(1, n, "f16", p)
    a, b, c = op(x, 1, 0), op(x, 1, 1), op(x, 2, 0)
    for t in (a, b, c):      # six standard deviations of the binomial
        assert abs(float((t == 0).float().mean()) - p) < 6 * math.sqrt(p * (1 - p) / n)
    assert abs(float(((a == 0) & (b == 0)).float().mean()) - p * p) < 1e-2 and not a.equal(b) and not a.equal(c)
    x[0, ::3] = float("nan")
    y = op(x, 1, 0)
    assert (y[a == 0] == 0).all()                                          # a dropped NaN is gone
    assert torch.equal(torch.isnan(y), torch.isnan(x) & (a != 0))
    assert op(x, 1, 0, y=x) is x and torch.equal(torch.nan_to_num(x, 5.0), torch.nan_to_num(y, 5.0))   # in place


def test_dropout_beyond_32_bit_indexes():
    import torch
    from dense_convolution_gb300 import head
    rows, cols, seed = 3, 2 ** 31 - 8, 12345
    x = torch.ones(rows, cols, device="cuda", dtype=torch.float16)
    y = head.Dropout(rows, cols, "f16", 0.5)(x, seed, 2, y=x)
    total, n = rows * cols, 4096                                           # the last n elements, n a multiple of 8
    low, first = np.uint64(0xFFFFFFFF), (total - n) // 8
    assert total % 8 == 0 and total > 2 ** 32
    i = np.arange(first, total // 8, dtype=np.uint64)
    c = [i & low, i >> np.uint64(32), np.full(i.size, 2, np.uint64), np.zeros(i.size, np.uint64)]
    k0, k1 = seed, 0
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = np.stack(c, 1)
    high = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)
    keep = torch.from_numpy(high >= 0x8000).cuda()                         # p = 1/2: the high half decides alone
    assert torch.equal(y.view(-1)[-n:] != 0, keep)


def test_dropout_index_does_not_depend_on_strides_or_types():
    import torch
    from dense_convolution_gb300 import head
    x = torch.ones(50, 40, device="cuda")
    a = head.Dropout(50, 40, "f32", 0.4)(x, 7, 9) == 0
    xs, _ = _strided(x.to(torch.bfloat16), 43, 1)
    b = head.Dropout(50, 40, "bf16", 0.4, x_stride=43)(xs, 7, 9) == 0
    c = head.Dropout(1, 2000, "f16", 0.4)(x.half().view(1, 2000), 7, 9).view(50, 40) == 0
    assert a.equal(b) and a.equal(c)


# ------------------------------------------------------------------ linear cross entropy
def _ce_inputs(seed, n, d, v, dtype, ignored=0.1, lean=3.0):
    import torch
    g = _gen(seed)
    w = (_randn(g, v, d) * (2.0 / math.sqrt(d))).to(_dt(dtype))
    target = torch.randint(0, v, (n,), generator=g, device="cuda")
    wy = w[target].float()
    h = (_randn(g, n, d) + lean * torch.rand(n, 1, generator=g, device="cuda") * wy / wy.norm(dim=1, keepdim=True).clamp_min(1e-6)).to(_dt(dtype))
    target[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    return h, w, target


def _ce_reference(h, w, target, reduction, dloss, ignore=-100):
    import torch
    h, w = h.double(), w.double()
    n, v = h.shape[0], w.shape[0]
    z = h @ w.T
    lse = torch.logsumexp(z, 1)
    live = (target != ignore) & (target >= 0) & (target < v)
    y = torch.where(live, target, 0)
    loss = torch.where(live, lse - z.gather(1, y[:, None])[:, 0], 0.0)
    count = live.sum().clamp_min(1)
    g = dloss.double().expand(n) / (count if reduction == "mean" else 1) * live
    p = torch.exp(z - lse[:, None])
    p[torch.arange(n, device="cuda"), y] -= 1.0
    dz = torch.where(live[:, None], p * g[:, None], 0.0)
    r = {"lse": lse, "z_size": (h.abs() @ w.abs().T).amax(1), "live": live,
         "loss": {"none": loss, "sum": loss.sum(), "mean": loss.sum() / count}[reduction],
         "dh": dz @ w, "dh_size": dz.abs() @ w.abs(), "dw": dz.T @ h, "dw_size": dz.abs().T @ h.abs()}
    # Before p - 1 cancels, what carries p's own error.
    p[torch.arange(n, device="cuda"), y] += 1.0
    pg = p * g.abs()[:, None]
    r["dh_p"], r["dw_p"] = pg @ w.abs(), pg.T @ h.abs()
    return r


def _check_ce(h, w, target, dtype, reduction, op, dloss, tag=""):
    import torch
    n, d = h.shape
    v = w.shape[0]
    r = _ce_reference(h, w, target, reduction, dloss)
    loss, lse = op(h, w, target)
    # z: 16 truncating steps (2 e) a segment, an addition a segment; fp32 parts add six products' worth.
    times = 6 if dtype == "f32" else 1
    z_tol = (32 + times * (d / 256 + 1) + (8 if dtype == "f32" else 0)) * E * r["z_size"] + 8 * E * r["lse"].abs() + 8 * E
    _close(lse, r["lse"], z_tol, tag + "lse")
    loss_tol = 2 * z_tol + 8 * E * (r["loss"].abs() if reduction == "none" else 0)
    if reduction != "none":
        loss_tol = loss_tol[r["live"]].sum() / (max(1, int(r["live"].sum())) if reduction == "mean" else 1) \
            + 64 * E * r["loss"].abs() + 1e-30
    _close(loss, r["loss"], loss_tol, tag + "loss")
    dh, dw = op.backward(h, w, target, lse, dloss)
    # p inherits z's and lse's absolute errors as a relative one, which p - 1 keeps
    # whole; then dz rounds (16 bits), and sums of K terms take K / 16 truncating steps.
    u = U[dtype] if dtype != "f32" else 8 * E
    p_tol = float(3 * z_tol.max()) + 8 * E
    steps_h = 2 * E * ((v / 16 + 64) if dtype != "f32" else 64 + 6 * v / 256)
    steps_w = 2 * E * ((n / 16 + 64) if dtype != "f32" else 64 + 6 * n / 256)
    _close(dh, r["dh"], U[dtype] * r["dh"].abs() + (u + steps_h) * r["dh_size"] + p_tol * r["dh_p"] + 1e-30, tag + "dh")
    _close(dw, r["dw"], U[dtype] * r["dw"].abs() + (u + steps_w) * r["dw_size"] + p_tol * r["dw_p"] + 1e-30, tag + "dw")
    for got, want in ((dh, r["dh"]), (dw, r["dw"])):
        norm = want.norm()
        if norm > 0 and want.numel() >= 1000:    # many independent roundings of dz and of the result: about 0.6 u each
            off = float((got.double() - want).norm() / norm)
            # (fp16: below 2^-14 the result's own rounding is up to 2^-25 whatever its size.)
            low = float((want.half().double() - want).norm() / norm) if dtype == "f16" else 0.0
            assert off < math.hypot(U[dtype] if dtype != "f32" else 64 * E, low), (tag, off, low)
    assert not dh[~r["live"]].any()
    return loss, lse, dh, dw


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v", [(1, 8, 1), (1, 1, 5), (1, 64, 1000), (2, 16, 33), (7, 24, 100), (128, 64, 256),
                                   (129, 72, 257), (300, 509, 1003), (1, 1024, 5000), (64, 256, 20000), (777, 130, 2011),
                                   (1000, 64, 63), (257, 8, 4000), (513, 640, 1537), (5, 4096, 300), (2500, 96, 70),
                                   (2000, 520, 30001), (1500, 1032, 9000), (8, 3801, 1500), (8, 4800, 700), (3, 320, 29888),
                                   (4, 2487, 2021), (16, 640, 3001), (11, 333, 2000), (1, 6144, 12345), (2, 31, 3), (6, 1, 9), (8, 1098, 5171)])
def test_linear_ce(dtype, n, d, v):
    import torch
    from dense_convolution_gb300 import head
    h, w, target = _ce_inputs(n * 31 + d * 7 + v, n, d, v, dtype)
    for reduction in ("none", "sum", "mean"):
        op = head.LinearCrossEntropy(n, d, v, dtype, reduction=reduction)
        dloss = torch.rand(n, device="cuda") + 0.5 if reduction == "none" else torch.full((), 0.7, device="cuda")
        _check_ce(h, w, target, dtype, reduction, op, dloss, reduction + " ")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_ce_pieces_agree(dtype):
    """The vocabulary in pieces (the last one short), and in one."""
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 200, 136, 2500
    h, w, target = _ce_inputs(4, n, d, v, dtype)
    dloss = torch.ones((), device="cuda")
    for piece in (256, 700, 1024, None):
        op = head.LinearCrossEntropy(n, d, v, dtype, piece=piece)
        _check_ce(h, w, target, dtype, "mean", op, dloss, f"piece {piece} ")


@pytest.mark.parametrize("dtype,hs,ws", [("bf16", 136, 144), ("f16", 131, 128), ("bf16", 128, 129), ("f32", 130, 131)])
def test_linear_ce_strides(dtype, hs, ws):
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 150, 128, 700
    h, w, target = _ce_inputs(9, n, d, v, dtype)
    hv, _ = _strided(h, hs)
    wv, _ = _strided(w, ws)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum", h_stride=hs, w_stride=ws)
    _check_ce(hv, wv, target, dtype, "sum", op, torch.ones((), device="cuda"))


@pytest.mark.parametrize("dtype,n,hs,ws", [("bf16", 1, 136, 144), ("f16", 3, 131, 129), ("bf16", 8, 128, 130),
                                           ("f32", 5, 130, 131), ("f32", 2, 132, 136)])
def test_linear_ce_few_tokens_strides(dtype, n, hs, ws):
    import torch
    from dense_convolution_gb300 import head
    d, v = 128, 700
    h, w, target = _ce_inputs(19, n, d, v, dtype, ignored=0.0)
    hv, _ = _strided(h, hs)
    wv, _ = _strided(w, ws)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="mean", h_stride=hs, w_stride=ws)
    _check_ce(hv, wv, target, dtype, "mean", op, torch.ones((), device="cuda"))


@pytest.mark.parametrize("n", [8, 140])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_ce_all_ignored_and_masked_nan(dtype, n):
    """Rows without a target: no loss, no gradient, whatever they hold."""
    import torch
    from dense_convolution_gb300 import head
    d, v = 64, 500
    h, w, target = _ce_inputs(2, n, d, v, dtype, ignored=0.0)
    one = torch.ones((), device="cuda")
    op = head.LinearCrossEntropy(n, d, v, dtype)
    none = torch.full_like(target, -100)
    loss, lse = op(h, w, none)
    assert float(loss) == 0.0 and torch.isfinite(lse).all()
    dh, dw = op.backward(h, w, none, lse, one)
    assert not dh.any() and not dw.any()
    target[::3] = -100
    loss0, lse0 = op(h, w, target)
    dh0, dw0 = op.backward(h, w, target, lse0, one)
    h2 = h.clone()
    h2[::3] = float("nan")
    h2[3] = float("inf")
    loss2, lse2 = op(h2, w, target)
    assert loss2.equal(loss0)
    dh2, dw2 = op.backward(h2, w, target, lse2, one)
    assert dh2.equal(dh0) and dw2.equal(dw0)


def test_linear_ce_target_out_of_range():
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 20, 32, 90
    h, w, target = _ce_inputs(6, n, d, v, "bf16", ignored=0.0)
    target[3], target[4] = v, -7
    rows = head.LinearCrossEntropy(n, d, v, "bf16", reduction="none")
    loss, lse = rows(h, w, target)
    assert torch.isnan(loss[[3, 4]]).all() and torch.isfinite(loss[[0, 1, 2, 5]]).all()
    dh, dw = rows.backward(h, w, target, lse, torch.ones(n, device="cuda"))
    assert not dh[[3, 4]].any() and torch.isfinite(dw.float()).all()
    assert torch.isnan(head.LinearCrossEntropy(n, d, v, "bf16")(h, w, target)[0])


def test_linear_ce_other_ignore_index():
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 33, 40, 64
    h, w, target = _ce_inputs(8, n, d, v, "f16", ignored=0.0)
    target[::2] = 0
    op = head.LinearCrossEntropy(n, d, v, "f16", reduction="none", ignore_index=0)
    loss, _ = op(h, w, target)
    assert (loss[target == 0] == 0).all() and (loss[target != 0] > 0).all()


def test_linear_ce_extreme_logits():
    """Logits far apart, and equal ones: the maximum is taken out first."""
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 130, 64, 1000
    for dtype in ("bf16", "f16", "f32"):
        h = torch.zeros(n, d, device="cuda", dtype=_dt(dtype))
        w = torch.zeros(v, d, device="cuda", dtype=_dt(dtype))
        h[:, 0] = 100.0
        w[:, 0] = torch.linspace(-100, 100, v, device="cuda")              # logits from -10^4 to 10^4
        h[1] = 0                                                           # all logits equal
        target = torch.full((n,), v - 1, device="cuda")
        target[2] = 0
        op = head.LinearCrossEntropy(n, d, v, dtype, reduction="none")
        loss, lse = op(h, w, target)
        z = (h.double() @ w.double().T)
        want = torch.logsumexp(z, 1)
        assert torch.allclose(lse.double(), want, rtol=1e-6, atol=1e-5)
        assert abs(float(loss[1]) - math.log(v)) < 1e-5
        assert abs(float(loss[2]) - float(want[2] - z[2, 0])) < 1e-2
        dh, dw = op.backward(h, w, target, lse, torch.ones(n, device="cuda"))
        assert torch.isfinite(dh.float()).all() and torch.isfinite(dw.float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_ce_tiny_upstream_gradients(dtype):
    """dloss far below fp16's range: it multiplies the fp32 result."""
    import torch
    from dense_convolution_gb300 import head
    n, d, v = 64, 64, 300
    h, w, target = _ce_inputs(12, n, d, v, dtype)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="sum")
    _, lse = op(h, w, target)
    big = op.backward(h, w, target, lse, torch.full((), 1.0, device="cuda"))
    if dtype == "bf16":
        small = op.backward(h, w, target, lse, torch.full((), 2.0 ** -40, device="cuda"))
        for a, b in zip(big, small):
            assert torch.equal(a.float() * 2.0 ** -40, b.float())
    rows = head.LinearCrossEntropy(n, d, v, dtype, reduction="none")
    up = rows.backward(h, w, target, lse, torch.full((n,), 2.0 ** 10, device="cuda"))
    for a, b in zip(big, up):
        normal = a.abs() >= 2.0 ** -14                                     # (below it fp16 has fewer bits)
        assert torch.equal(a.float()[normal] * 2.0 ** 10, b.float()[normal])


@pytest.mark.parametrize("n,d,v", [(40, 32, 150), (300, 520, 1100), (7, 33, 150), (16, 100, 333)])
def test_linear_ce_gradient_against_differences(n, d, v):
    """fp32: the loss's difference along a direction is the gradient's part of it."""
    import torch
    from dense_convolution_gb300 import head
    h, w, target = _ce_inputs(21, n, d, v, "f32")
    g = _gen(1)
    dhdir, dwdir = _randn(g, n, d), _randn(g, v, d) / math.sqrt(d)
    op = head.LinearCrossEntropy(n, d, v, "f32", reduction="none")
    weight = torch.rand(n, generator=g, device="cuda") + 0.5
    val = lambda h, w: (op(h, w, target)[0].double() * weight.double()).sum()
    _, lse = op(h, w, target)
    dh, dw = op.backward(h, w, target, lse, weight)
    s = 1e-2
    tol = 2e-3 * math.sqrt(n)
    assert abs(float((val(h + s * dhdir, w) - val(h - s * dhdir, w)) / (2 * s) - (dh.double() * dhdir).sum())) < tol
    assert abs(float((val(h, w + s * dwdir) - val(h, w - s * dwdir)) / (2 * s) - (dw.double() * dwdir).sum())) < tol


@pytest.mark.parametrize("n,d,dtype", [(300, 264, "bf16"), (8, 264, "bf16"), (1, 1001, "f16"), (13, 130, "f32")])
def test_linear_ce_is_repeatable_and_keeps_to_its_buffers(n, d, dtype):
    import torch
    from dense_convolution_gb300 import head, head_capi
    v = 3000
    h, w, target = _ce_inputs(30, n, d, v, dtype)
    op = head.LinearCrossEntropy(n, d, v, dtype, reduction="none", piece=1024)
    dloss = torch.rand(n, device="cuda")
    first = None
    for fill in (0x00, 0xFF, 0x7F):                                        # whatever the workspace held
        f = torch.full((op.workspace_bytes + 4096,), fill, dtype=torch.uint8, device="cuda")
        b = torch.full((op.backward_workspace_bytes + 4096,), fill, dtype=torch.uint8, device="cuda")
        loss, lse = op(h, w, target, workspace=f[:op.workspace_bytes])
        dh, dw = op.backward(h, w, target, lse, dloss, workspace=b[:op.backward_workspace_bytes])
        assert (f[op.workspace_bytes:] == fill).all() and (b[op.backward_workspace_bytes:] == fill).all()
        out = [t.clone() for t in (loss, lse, dh, dw)]
        if first is None:
            first = out
        assert all(p.equal(q) for p, q in zip(first, out))
    only_h, none = op.backward(h, w, target, lse, dloss, need_dw=False)
    assert none is None and only_h.equal(first[2])
    none, only_w = op.backward(h, w, target, lse, dloss, need_dh=False)
    assert none is None and only_w.equal(first[3])


@pytest.mark.parametrize("n", [2, 20])
def test_linear_ce_beyond_32_bit_offsets(n):
    """A vocabulary whose weights pass 2^32 elements: all zero but for the first and last rows."""
    import torch
    from dense_convolution_gb300 import head
    d, v, k = 4096, 2 ** 20 + 5, 3
    g = _gen(n)
    ends = (_randn(g, 2 * k, d) * (2.0 / math.sqrt(d))).to(torch.bfloat16)
    w = torch.zeros(v, d, device="cuda", dtype=torch.bfloat16)
    w[:k], w[-k:] = ends[:k], ends[k:]
    h = (_randn(g, n, d) + 3 * ends[-1].float() / ends[-1].float().norm()).to(torch.bfloat16)
    target = torch.full((n,), v - 1, device="cuda")
    target[1] = 1
    op = head.LinearCrossEntropy(n, d, v, "bf16", reduction="sum")
    loss, lse = op(h, w, target)
    dh, dw = op.backward(h, w, target, lse, torch.ones((), device="cuda"))
    z = h.double() @ ends.double().T
    want = torch.log((v - 2 * k) + z.exp().sum(1))
    # v sums of about 1 each in fp32, joined by trees and chains of a few hundred
    _close(lse, want, 512 * E * want.abs(), "lse")
    y = torch.full((n,), 2 * k - 1, device="cuda")
    y[1] = 1
    _close(loss, (want - z.gather(1, y[:, None])[:, 0]).sum(), n * 512 * E * want.abs().max() + 64 * E * z.abs().max(), "loss")
    p = torch.exp(z - want[:, None])
    p[torch.arange(n, device="cuda"), y] -= 1.0
    dh_want, size = p @ ends.double(), p.abs() @ ends.double().abs()
    _close(dh, dh_want, U["bf16"] * dh_want.abs() + (U["bf16"] + 1e-4) * size + 1e-30, "dh")
    dw_want, size = p.T @ h.double(), p.T.abs() @ h.double().abs()
    got = torch.cat([dw[:k], dw[-k:]])
    _close(got, dw_want, U["bf16"] * dw_want.abs() + (U["bf16"] + 1e-4) * size + 1e-30, "dw")
    middle = torch.exp(-want)[:, None].expand(n, 1).T @ h.double()         # every other row: p = exp(-lse)
    size = torch.exp(-want)[None] @ h.double().abs()
    for row in (k, v // 2, v - k - 1):
        _close(dw[row:row + 1], middle, U["bf16"] * middle.abs() + (U["bf16"] + 1e-4) * size + 1e-30, f"dw {row}")


def test_linear_ce_no_tokens():
    import torch
    from dense_convolution_gb300 import head
    op = head.LinearCrossEntropy(0, 16, 50, "bf16")
    h, w = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16), torch.ones(50, 16, device="cuda", dtype=torch.bfloat16)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = op(h, w, t)
    assert float(loss) == 0.0 and lse.shape == (0,)
    dh, dw = op.backward(h, w, t, lse, torch.ones((), device="cuda"))
    assert dh.shape == (0, 16) and not dw.any()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("n", [256, 6])
def test_other_stream_and_capture(n):
    """The operators on a stream that is not the tensors' own, and in a graph."""
    import torch
    from dense_convolution_gb300 import head
    d, v = 512, 1500
    h, w, target = _ce_inputs(40, n, d, v, "bf16")
    gamma, beta = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    ln = head.LayerNorm(n, d, "bf16", "f32")
    dr = head.Dropout(n, d, "bf16", 0.2)
    ce = head.LinearCrossEntropy(n, d, v, "bf16")
    one = torch.ones((), device="cuda")

    def step(stream=None):
        y, mean, rstd = ln(h, gamma, beta, stats=True, stream=stream)
        z = dr(y, 11, 5, stream=stream)
        loss, lse = ce(z, w, target, stream=stream)
        dz, dw = ce.backward(z, w, target, lse, one, stream=stream)
        dy = dr.backward(dz, 11, 5, stream=stream)
        return [loss, dw, *ln.backward(dy, h, gamma, mean, rstd, stream=stream)]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(a.equal(b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(a.equal(b) for a, b in zip(want, captured))


def test_wrong_tensors_are_refused():
    import torch
    from dense_convolution_gb300 import head
    x = torch.zeros(4, 8, device="cuda")
    ln, dr, ce = head.LayerNorm(4, 8), head.Dropout(4, 8), head.LinearCrossEntropy(4, 8, 16, "f32")
    for bad in (x.half(), x[:, :7], x.T.contiguous(), x.cpu(), torch.zeros(4, 16, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            ln(bad)
        with pytest.raises(ValueError):
            dr(bad, 1)
        with pytest.raises(ValueError):
            ce(bad, torch.zeros(16, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ln(x, torch.ones(8, device="cuda").half())
    with pytest.raises(ValueError):
        ce(x, torch.zeros(16, 8, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        head.LayerNorm(8, 4, pixels=4)(torch.zeros(2, 5, 4, device="cuda"))


def test_waits_that_run_out_are_reported():
    """A limit of a nanosecond makes the kernels' ordinary waits give up: the
    status says so, and the next call under the default limit is right."""
    import torch
    from dense_convolution_gb300 import capi, head
    n, d, v = 600, 1024, 2000
    h, w, target = _ce_inputs(50, n, d, v, "bf16")
    x = _randn(_gen(2), 4000, 2048).to(torch.bfloat16)
    planes = _randn(_gen(3), 8, 256, 400).to(torch.bfloat16)
    ce, ln = head.LinearCrossEntropy(n, d, v, "bf16"), head.LayerNorm(4000, 2048, "bf16", "f32")
    pl = head.LayerNorm(3200, 256, "bf16", "f32", pixels=400)

    def calls():
        loss, _ = ce(h, w, target)
        _, mean, rstd = ln(x, stats=True)
        dx, _, _ = ln.backward(x, x, None, mean, rstd)
        return [loss, dx, pl(planes)]

    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    try:
        capi.conv2d_set_wait_limit(1, stream)
        calls()
        torch.cuda.synchronize()
        assert capi.conv2d_device_status(stream) != 0
    finally:
        capi.conv2d_set_wait_limit(0, stream)
    capi.conv2d_device_status(stream)
    assert all(a.equal(b) for a, b in zip(want, calls()))
