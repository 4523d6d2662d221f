"""The operators of a training head on convolution features, as measured cases.

A frozen convolution trunk gives features; layer norm turns them into token
rows, dropout (with a residual) regularises them, and the linear cross entropy
scores every token against a vocabulary and returns the gradients.  Each
operator is given here in a plain form (elementary torch operations in 32 bits,
rounded once at the end), as the calls a user makes of the package (`own`), and
once more from its definition in 64 bits (`exact`).

    layer norm      y = (x - mean) rstd gamma + beta over each row, and from dy:
                    dx, dgamma, dbeta.  x is rows of columns (any row stride),
                    or channels-first planes [image][channel][pixel], one row a
                    pixel.
    dropout         y = residual + keep x / (1 - p), dx = keep dy / (1 - p).
                    keep of element i (row-major index) comes from Philox4x32-10
                    ("Parallel random numbers: as easy as 1, 2, 3", 2011): word
                    i%8 of the 16-bit words of Philox(seed; i/8, offset) is the
                    high half of a 32-bit number, the same word of the stream
                    whose last counter bit is set the low half; an element is
                    dropped where that number is below round(p 2^32).
    linear_ce       loss_n = logsumexp_v(h_n . w_v) - h_n . w_target, zero for
                    ignored targets; reduced by none, sum or mean over the
                    targets that count; dh and dw from the loss's gradient.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-5
_IGNORE = -100


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a serving step: the launch is all that counts.
        {"name": "norm_one_token", "op": "norm", "dir": "fwd", "dtype": "bf16", "param": "bf16", "images": 0,
         "rows": 1, "cols": 4096, "gap": 0},
        # The backward pass of a training batch: 16384 tokens, bf16 activations, fp32 parameters.
        {"name": "norm_train_rows", "op": "norm", "dir": "bwd", "dtype": "bf16", "param": "f32", "images": 0,
         "rows": 16384, "cols": 2048, "gap": 0},
        # Odd rows inside a wider buffer (a slice of a concatenated projection), both directions, fp32.
        {"name": "norm_odd_slice", "op": "norm", "dir": "step", "dtype": "f32", "param": "f32", "images": 0,
         "rows": 1537, "cols": 771, "gap": 5},
        # The features of the 512-channel 28x28 layer at batch 64, normalised over channels into token rows, trained.
        {"name": "norm_features", "op": "norm", "dir": "step", "dtype": "bf16", "param": "f32", "images": 64,
         "rows": 64 * 784, "cols": 512, "gap": 0},
        # Whole images of the 64-channel 56x56 layer normalised at once: few, very long rows.
        {"name": "norm_whole_images", "op": "norm", "dir": "fwd", "dtype": "f16", "param": "f16", "images": 0,
         "rows": 32, "cols": 64 * 56 * 56, "gap": 0},
        # Dropout on a training batch, joined with the residual stream.
        {"name": "drop_residual", "op": "drop", "dir": "fwd", "dtype": "bf16", "rows": 16384, "cols": 2048, "gap": 0,
         "p": 0.1, "residual": True},
        # A few odd rows, both directions: the smallest call.
        {"name": "drop_small_odd", "op": "drop", "dir": "step", "dtype": "f32", "rows": 7, "cols": 1001, "gap": 0,
         "p": 0.5, "residual": False},
        # The loss of one new token: one pass over the vocabulary's weights.
        {"name": "ce_one_token", "op": "ce", "dir": "fwd", "dtype": "bf16", "tokens": 1, "hidden": 1024,
         "vocab": 32000, "reduction": "none", "ignored": 0.0},
        # Scoring a held-out batch: the loss of every token, no gradients.
        {"name": "ce_score", "op": "ce", "dir": "fwd", "dtype": "bf16", "tokens": 8192, "hidden": 1024,
         "vocab": 32768, "reduction": "none", "ignored": 0.1},
        # A full training step over a large vocabulary: the largest case.
        {"name": "ce_train", "op": "ce", "dir": "step", "dtype": "bf16", "tokens": 8192, "hidden": 2048,
         "vocab": 131072, "reduction": "mean", "ignored": 0.05},
        # A ragged step: token, feature and vocabulary counts that fit no tile, many targets masked.
        {"name": "ce_train_ragged", "op": "ce", "dir": "step", "dtype": "f16", "tokens": 777, "hidden": 509,
         "vocab": 10007, "reduction": "mean", "ignored": 0.4},
        # The same in fp32, for runs that keep their head in full precision.
        {"name": "ce_train_f32", "op": "ce", "dir": "step", "dtype": "f32", "tokens": 1000, "hidden": 768,
         "vocab": 20011, "reduction": "sum", "ignored": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over its logarithm; half of them multiples of 64 where they can be."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "drop", "ce", "ce"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        form = rng.choice(["rows", "rows", "planes", "long"])
        c = {"op": "norm", "dir": rng.choice(["fwd", "bwd", "step"]), "dtype": dtype,
             "param": rng.choice([dtype, "f32"]), "images": 0, "gap": 0}
        if form == "planes":
            c["images"] = _log(rng, 1, 64)
            side = _log(rng, 3, 56)
            c["rows"] = c["images"] * side * side
            c["cols"] = _size(rng, 16, max(16, min(1024, (64 * 784 * 512) // c["rows"])))
        elif form == "long":
            c["rows"] = _log(rng, 1, 32)
            c["cols"] = _log(rng, 20000, 64 * 56 * 56)
        else:
            c["cols"] = _size(rng, 64, 16384)
            c["rows"] = _log(rng, 1, max(1, min(65536, (16384 * 2048) // c["cols"])))
            c["gap"] = rng.choice([0, 0, 8, rng.randint(1, 64)])
        return c
    if op == "drop":
        cols = _size(rng, 16, 16384)
        return {"op": "drop", "dir": rng.choice(["fwd", "bwd", "step"]), "dtype": dtype,
                "rows": _log(rng, 1, max(1, (16384 * 2048) // cols)), "cols": cols,
                "gap": rng.choice([0, 0, 8, rng.randint(1, 64)]), "p": rng.choice([0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)]),
                "residual": rng.random() < 0.5}
    most = 2.0e10 if dtype == "f32" else 2.0e12          # tokens * hidden * vocab
    hidden = _size(rng, 64, 4096)
    vocab = _size(rng, 1000, 131072)
    tokens = _log(rng, 1, int(max(1, min(8192, most / (hidden * vocab)))))
    return {"op": "ce", "dir": rng.choice(["fwd", "step", "step"]), "dtype": dtype, "tokens": tokens, "hidden": hidden,
            "vocab": vocab, "reduction": rng.choice(["none", "sum", "mean"]), "ignored": rng.choice([0.0, 0.1, 0.5])}


# ------------------------------------------------------------------ inputs
def _rows(gen, rows, cols, gap, dtype, scale=1.0, mean=0.0):
    """Activations: a slice of a buffer whose rows are `gap` elements longer."""
    t = torch.randn(rows, cols + gap, generator=gen, device="cuda", dtype=torch.float32)
    return (t * scale + mean).to(dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = _DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        rows, cols, images = case["rows"], case["cols"], case["images"]
        pt = _DT[case["param"]]
        if images:
            # Convolution outputs: channels with offsets of their own.
            off = torch.randn(1, cols, 1, generator=gen, device="cuda") * 0.5 + 0.3
            s["x"] = (torch.randn(images, cols, rows // images, generator=gen, device="cuda") + off).to(dt)
        else:
            s["x"] = _rows(gen, rows, cols, case["gap"], dt, 1.5, 0.4)
        s["gamma"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(pt)
        s["beta"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(pt)
        if case["dir"] != "fwd":
            s["dy"] = torch.randn(rows, cols, generator=gen, device="cuda").to(dt)
        if case["dir"] == "bwd":
            # What the forward pass of this step left behind.
            x = _as_rows(case, s["x"]).double()
            var, mean = torch.var_mean(x, dim=1, correction=0)
            s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + _EPS).float()
        if own:
            from dense_convolution_gb300 import head
            s["op"] = head.LayerNorm(rows, cols, case["dtype"], case["param"], eps=_EPS,
                                     pixels=rows // images if images else None,
                                     x_stride=None if images else cols + case["gap"])
    elif case["op"] == "drop":
        s["x"] = _rows(gen, case["rows"], case["cols"], case["gap"], dt)
        s["residual"] = _rows(gen, case["rows"], case["cols"], 0, dt, 2.0) if case["residual"] else None
        s["dy"] = _rows(gen, case["rows"], case["cols"], 0, dt) if case["dir"] != "fwd" else None
        # The generator's state: a run's seed, and the draws made before this call.
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ (int(seed) * 0x2545F4914F6CDD1D % 2 ** 64), 41 + int(seed) % 1000
        if own:
            from dense_convolution_gb300 import head
            s["op"] = head.Dropout(case["rows"], case["cols"], case["dtype"], case["p"],
                                   x_stride=case["cols"] + case["gap"])
    else:
        n, d, v = case["tokens"], case["hidden"], case["vocab"]
        s["w"] = (torch.randn(v, d, generator=gen, device="cuda") * (2.0 / math.sqrt(d))).to(dt)
        # Word frequencies fall off as a power of the rank.
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        s["target"] = (v ** u - 1.0).long().clamp_(0, v - 1)
        # A partly trained model: every token leans towards its target, some strongly.
        lean = torch.rand(n, 1, generator=gen, device="cuda") * 5.0
        wy = s["w"][s["target"]].float()
        h = torch.randn(n, d, generator=gen, device="cuda")
        s["h"] = (h + lean * wy / wy.norm(dim=1, keepdim=True).clamp_min(1e-6)).to(dt)
        s["target"][torch.rand(n, generator=gen, device="cuda") < case["ignored"]] = _IGNORE
        if case["dir"] == "step":
            s["dloss"] = (torch.rand(n, generator=gen, device="cuda") + 0.5) if case["reduction"] == "none" \
                else torch.full((), 1.0, device="cuda")
        if own:
            from dense_convolution_gb300 import head
            s["op"] = head.LinearCrossEntropy(n, d, v, case["dtype"], reduction=case["reduction"],
                                              ignore_index=_IGNORE)
    return s


def _as_rows(case, x):
    """[image][channel][pixel] planes as rows of channels."""
    return x.transpose(1, 2).reshape(case["rows"], case["cols"]) if case["images"] else x


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _plain_norm, "drop": _plain_drop, "ce": _plain_ce}[c["op"]](s, c)


def _run_own(s, c):
    op = s["op"]
    out = {}
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            return {"y": op(s["x"], s["gamma"], s["beta"])}
        if c["dir"] == "step":
            out["y"], out["mean"], out["rstd"] = op(s["x"], s["gamma"], s["beta"], stats=True)
            mean, rstd = out["mean"], out["rstd"]
        else:
            mean, rstd = s["mean"], s["rstd"]
        out["dx"], out["dgamma"], out["dbeta"] = op.backward(s["dy"], s["x"], s["gamma"], mean, rstd)
    elif c["op"] == "drop":
        if c["dir"] != "bwd":
            out["y"] = op(s["x"], s["seed"], s["offset"], residual=s["residual"])
        if c["dir"] != "fwd":
            out["dx"] = op.backward(s["dy"], s["seed"], s["offset"])
    else:
        loss, lse = op(s["h"], s["w"], s["target"])
        out["loss"], out["lse"] = loss, lse
        if c["dir"] == "step":
            out["dh"], out["dw"] = op.backward(s["h"], s["w"], s["target"], lse, s["dloss"])
    return out


# ------------------------------------------------------------------ plain forms (32 bits)
def _plain_norm(s, c):
    dt, pt = _DT[c["dtype"]], _DT[c["param"]]
    x = _as_rows(c, s["x"]).float()
    gamma, beta = s["gamma"].float(), s["beta"].float()
    out = {}
    if c["dir"] == "bwd":
        mean, rstd = s["mean"], s["rstd"]
    else:
        mean = x.mean(dim=1)
        centred = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((centred * centred).mean(dim=1) + _EPS)
        out["y"] = (centred * rstd[:, None] * gamma + beta).to(dt)
        if c["dir"] == "fwd":
            return out
        out["mean"], out["rstd"] = mean, rstd
    dy = s["dy"].float()
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = ((g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True)) * rstd[:, None]).to(dt)
    if c["images"]:
        dx = dx.reshape(c["images"], -1, c["cols"]).transpose(1, 2).contiguous()
    out["dx"], out["dgamma"], out["dbeta"] = dx, (dy * xhat).sum(dim=0).to(pt), dy.sum(dim=0).to(pt)
    return out


_M = 0xFFFFFFFF


def _philox_words(seed, offset, blocks, stream):
    """The four 32-bit words of each of the first `blocks` counters, as int64."""
    i = torch.arange(blocks, device="cuda", dtype=torch.int64)
    c0, c1 = i & _M, i >> 32
    c2 = torch.full_like(i, offset & _M)
    c3 = torch.full_like(i, (offset >> 32) | (stream << 31))
    k0, k1 = seed & _M, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # the low 64 bits, wrapped
        c0, c1, c2, c3 = ((p1 >> 32) & _M) ^ c1 ^ k0, p1 & _M, ((p0 >> 32) & _M) ^ c3 ^ k1, p0 & _M
        k0, k1 = (k0 + 0x9E3779B9) & _M, (k1 + 0xBB67AE85) & _M
    return torch.stack([c0, c1, c2, c3], dim=1)


def _plain_keep(s, c):
    n = c["rows"] * c["cols"]
    blocks = (n + 7) // 8
    halves = []
    for stream in (0, 1):
        w = _philox_words(s["seed"], s["offset"], blocks, stream)
        halves.append(torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:n])
    return ((halves[0] << 16 | halves[1]) >= int(round(c["p"] * 2 ** 32))).reshape(c["rows"], c["cols"])


def _plain_drop(s, c):
    dt = _DT[c["dtype"]]
    keep = _plain_keep(s, c)
    scale = 1.0 / (1.0 - c["p"])
    out = {}
    if c["dir"] != "bwd":
        y = torch.where(keep, s["x"].float() * scale, 0.0)
        out["y"] = (y + s["residual"].float() if c["residual"] else y).to(dt)
    if c["dir"] != "fwd":
        out["dx"] = torch.where(keep, s["dy"].float() * scale, 0.0).to(dt)
    return out


def _plain_ce(s, c):
    h, w, target = s["h"].float(), s["w"].float(), s["target"]
    logits = h @ w.T
    counts = target != _IGNORE
    y = torch.where(counts, target, 0)
    top = logits.amax(dim=1)
    lse = top + (logits - top[:, None]).exp().sum(dim=1).log()
    per = torch.where(counts, lse - logits.gather(1, y[:, None])[:, 0], 0.0)
    number = counts.sum().clamp_min(1).float()
    loss = {"none": lambda: per, "sum": lambda: per.sum(), "mean": lambda: per.sum() / number}[c["reduction"]]()
    out = {"loss": loss, "lse": lse}
    if c["dir"] == "step":
        per_row = s["dloss"] / number if c["reduction"] == "mean" else s["dloss"]
        g = torch.where(counts, per_row, 0.0)
        p = logits.sub_(lse[:, None]).exp_()
        p[torch.arange(c["tokens"], device="cuda"), y] -= 1.0
        p *= g[:, None]
        out["dh"], out["dw"] = (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)
    return out


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "drop":
        return _exact_drop(s, case)
    # Three products of 2 tokens hidden vocab operations at about 1 TFLOP/s.
    if case["tokens"] * case["hidden"] * case["vocab"] * (6 if case["dir"] == "step" else 2) > 1.4e13:
        return None
    return _exact_ce(s, case)


def _exact_norm(s, c):
    x = s["x"].to(torch.float64)
    axis = 1                                               # columns, or channels of [image][channel][pixel]
    shape = (1, -1, 1) if c["images"] else (1, -1)
    gamma, beta = s["gamma"].to(torch.float64).view(shape), s["beta"].to(torch.float64).view(shape)
    n = c["cols"]

    def flat(t):                                           # planes to token rows
        return torch.movedim(t, 1, -1).reshape(c["rows"], n) if c["images"] else t

    if c["dir"] == "bwd":
        per = (c["images"], 1, -1) if c["images"] else (-1, 1)
        mu, r = s["mean"].to(torch.float64).view(per), s["rstd"].to(torch.float64).view(per)
    else:
        mu = x.sum(axis, keepdim=True) / n
        r = ((x - mu).square().sum(axis, keepdim=True) / n + _EPS).pow(-0.5)
    z = (x - mu) * r
    out = {}
    if c["dir"] != "bwd":
        out["y"] = flat(z * gamma + beta)
        if c["dir"] == "fwd":
            return out
        out["mean"], out["rstd"] = mu.reshape(-1), r.reshape(-1)
    dy = s["dy"].to(torch.float64)
    if c["images"]:
        dy = torch.movedim(dy.view(c["images"], -1, n), -1, 1)
    a = dy * gamma
    out["dx"] = r * (a - (a.sum(axis, keepdim=True) + z * (a * z).sum(axis, keepdim=True)) / n)
    rest = (0, 2) if c["images"] else (0,)
    out["dgamma"], out["dbeta"] = (dy * z).sum(rest), dy.sum(rest)
    return out


def _exact_drop(s, c):
    n = c["rows"] * c["cols"]
    number = np.zeros(-(-n // 8) * 8, dtype=np.uint32)
    low = np.uint64(_M)
    for part in (0, 1):
        x = np.zeros((4, number.size // 8), dtype=np.uint64)
        x[0] = np.arange(x.shape[1], dtype=np.uint64)      # fewer than 2^32 counters
        x[2], x[3] = s["offset"] % 2 ** 32, s["offset"] // 2 ** 32 + part * 2 ** 31
        key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
        for r in range(10):
            a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            ka, kb = (np.uint64((key[0] + r * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + r * 0xBB67AE85) % 2 ** 32))
            x = np.stack([(b >> np.uint64(32)) ^ x[1] ^ ka, b & low, (a >> np.uint64(32)) ^ x[3] ^ kb, a & low])
        words = np.ascontiguousarray(x.T.astype("<u4")).view("<u2").reshape(-1)
        number |= words.astype(np.uint32) << np.uint32(0 if part else 16)
    drop = torch.from_numpy(number[:n].astype(np.int64)).cuda().view(c["rows"], c["cols"]) < int(round(c["p"] * 2 ** 32))
    out = {}
    if c["dir"] != "bwd":
        y = s["x"].to(torch.float64) / (1.0 - c["p"])
        y[drop] = 0.0
        out["y"] = y + s["residual"].to(torch.float64) if c["residual"] else y
    if c["dir"] != "fwd":
        dx = s["dy"].to(torch.float64) / (1.0 - c["p"])
        dx[drop] = 0.0
        out["dx"] = dx
    return out


def _exact_ce(s, c):
    h, w, target = s["h"].to(torch.float64), s["w"].to(torch.float64), s["target"]
    live = torch.nonzero(target != _IGNORE)[:, 0]
    z = torch.mm(h, w.t())
    lse = torch.logsumexp(z, 1)
    loss = torch.zeros(c["tokens"], dtype=torch.float64, device="cuda")
    loss[live] = lse[live] - z[live, target[live]]
    n = max(1, live.numel())
    out = {"loss": {"none": loss, "sum": loss.sum(), "mean": loss.sum() / n}[c["reduction"]], "lse": lse}
    if c["dir"] == "step":
        weight = torch.zeros_like(loss)
        weight[live] = s["dloss"].to(torch.float64)[live] if c["reduction"] == "none" else s["dloss"].to(torch.float64)
        if c["reduction"] == "mean":
            weight /= n
        z = torch.softmax(z, 1)
        z[live, target[live]] -= 1.0
        z *= weight[:, None]
        out["dh"], out["dw"] = torch.mm(z, w), torch.mm(z.t(), h)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    e = size[case["dtype"]]
    if case["op"] == "norm":
        n, cols = case["rows"] * case["cols"], case["cols"]
        pe = size[case["param"]]
        fwd = {"bytes": 2 * n * e + 2 * cols * pe, "flops": 8 * n}
        bwd = {"bytes": 3 * n * e + 8 * case["rows"] + 3 * cols * pe, "flops": 14 * n}
        if case["dir"] == "fwd":
            return fwd
        if case["dir"] == "bwd":
            return bwd
        # x, dy, y and dx once each, the statistics written, gamma and beta read, their gradients written.
        return {"bytes": 4 * n * e + 8 * case["rows"] + 4 * cols * pe, "flops": 22 * n}
    if case["op"] == "drop":
        n = case["rows"] * case["cols"]
        b = 0
        if case["dir"] != "bwd":
            b += (3 if case["residual"] else 2) * n * e
        if case["dir"] != "fwd":
            b += 2 * n * e
        return {"bytes": b, "flops": (2 if case["dir"] == "step" else 1) * 2 * n}
    n, d, v = case["tokens"], case["hidden"], case["vocab"]
    rows = {"none": n, "sum": 1, "mean": 1}[case["reduction"]]
    if case["dir"] == "fwd":
        return {"bytes": (n * d + v * d) * e + 8 * n + 4 * n + 4 * rows, "flops": 2 * n * d * v}
    return {"bytes": 2 * (n * d + v * d) * e + 8 * n + 4 * n + 8 * rows, "flops": 6 * n * d * v}
