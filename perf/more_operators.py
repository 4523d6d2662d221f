"""The feed-forward block of a training head and the step that trains it, as measured cases.

Between the layer norm and the loss of a head on convolution features stands a
gated feed-forward block; AdamW turns the gradients of the whole head into its
next weights.  Each operator is given here in a plain form (elementary torch
operations in 32 bits, rounded once at the end), as the calls a user makes of
the package (`own`), and once more from its definition in 64 bits (`exact`).

    ffn     g = x wg', u = x wu', h = act(g) u, y = residual + h wd'; from dy:
            dx, dwg, dwu, dwd.  x is rows of `hidden` columns (any row stride),
            wg and wu [inner][hidden], wd [hidden][inner].  act(g) is
            g / (1 + exp(-g)) (silu), g Phi(g) (gelu) or its form by tanh.
    adamw   over many tensors, in place:
            m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
            p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps),
            and a 16-bit copy of p.  The moments of all tensors lie one tensor
            after the other, each padded to blocks of 256.  In 32 bits, or in 8:
            m in e4m3 and v in e5m2, each block times a power of two that takes
            its largest value to the type's top binade (at most 1.75 there).
            What 8 bits cannot hold goes to one of its neighbours with the
            chances that keep the mean: the low (m) and high (v) 16 bits of word
            i%4 of Philox4x32-10(seed; i/4, tensor, step) are added below the
            kept bits, for element i of a tensor.  A v above zero is never
            stored as zero.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = 256
_B1, _B2, _EPS, _LR = 0.9, 0.95, 1e-8, 1e-3

# The filters of the twelve layers of the convolution benchmark.
_FILTERS = "34848,34848,9408,9408,614400,1179648,1728,73728,36864,147456,589824,2359296"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a serving step: one pass over the block's weights.
        {"name": "ffn_one_token", "op": "ffn", "dir": "fwd", "dtype": "bf16", "act": "silu", "tokens": 1,
         "hidden": 2048, "inner": 8192, "gap": 0, "residual": True},
        # Sixteen sequences served together, a token each.
        {"name": "ffn_few_tokens", "op": "ffn", "dir": "fwd", "dtype": "f16", "act": "silu", "tokens": 16,
         "hidden": 4096, "inner": 16384, "gap": 0, "residual": True},
        # Scoring a held-out batch: no gradients, nothing kept.
        {"name": "ffn_score", "op": "ffn", "dir": "fwd", "dtype": "bf16", "act": "gelu", "tokens": 8192,
         "hidden": 1024, "inner": 4096, "gap": 0, "residual": True},
        # A training step of the block over a long batch: the most arithmetic.
        {"name": "ffn_train", "op": "ffn", "dir": "step", "dtype": "bf16", "act": "silu", "tokens": 8192,
         "hidden": 2048, "inner": 8192, "gap": 0, "residual": True},
        # The pixels of the 512-channel 28x28 layer at batch 64 as tokens, trained: many rows, few columns.
        {"name": "ffn_features", "op": "ffn", "dir": "step", "dtype": "bf16", "act": "gelu_tanh", "tokens": 64 * 784,
         "hidden": 512, "inner": 1408, "gap": 0, "residual": False},
        # A ragged step: counts that fit no tile, rows inside a wider buffer.
        {"name": "ffn_train_ragged", "op": "ffn", "dir": "step", "dtype": "f16", "act": "gelu", "tokens": 777,
         "hidden": 509, "inner": 1371, "gap": 3, "residual": True},
        # The same in fp32, for runs that keep their head in full precision.
        {"name": "ffn_train_f32", "op": "ffn", "dir": "step", "dtype": "f32", "act": "silu", "tokens": 1000,
         "hidden": 768, "inner": 2048, "gap": 0, "residual": True},
        # The gains and offsets of a few norms: the smallest step, where the launch is all.
        {"name": "adam_norms", "op": "adam", "grad": "f32", "copy": "", "states": "f32",
         "tensors": "512,512,2048,2048,64,64", "scale": False},
        # The convolution benchmark's filters, fine-tuned in full precision.
        {"name": "adam_filters", "op": "adam", "grad": "f32", "copy": "f16", "states": "f32", "tensors": _FILTERS,
         "scale": True},
        # A whole head: a vocabulary of 131072 by 2048, a block and its norm; bf16 gradients and copies.
        {"name": "adam_head", "op": "adam", "grad": "bf16", "copy": "bf16", "states": "f32",
         "tensors": "268435456,16777216,16777216,16777216,2048,2048", "scale": True},
        # The same with its moments in 8 bits.
        {"name": "adam_head_8bit", "op": "adam", "grad": "bf16", "copy": "bf16", "states": "8bit",
         "tensors": "268435456,16777216,16777216,16777216,2048,2048", "scale": True},
        # Many tensors of odd sizes, as low-rank adapters and biases have.
        {"name": "adam_odd_8bit", "op": "adam", "grad": "f16", "copy": "f16", "states": "8bit",
         "tensors": ",".join(str(1 + 3 * i + 97 * i * i) for i in range(90)), "scale": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over its logarithm; half of them multiples of 64 where they can be."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    if rng.random() < 0.6:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 8.0e9 if dtype == "f32" else 1.3e11          # tokens * hidden * inner
        hidden, inner = _size(rng, 64, 4096), _size(rng, 64, 16384)
        tokens = _log(rng, 1, int(max(1, min(50176, most / (hidden * inner)))))
        return {"op": "ffn", "dir": rng.choice(["fwd", "step", "step"]), "dtype": dtype,
                "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), "tokens": tokens, "hidden": hidden,
                "inner": inner, "gap": rng.choice([0, 0, 8, rng.randint(1, 64)]), "residual": rng.random() < 0.5}
    count, left = _log(rng, 1, 200), 1 << 27
    sizes = []
    for _ in range(count):
        sizes.append(_size(rng, 1, max(1, min(left, 1 << 26))))
        left = max(1, left - sizes[-1])
    return {"op": "adam", "grad": rng.choice(["bf16", "f16", "f32"]), "copy": rng.choice(["", "bf16", "f16"]),
            "states": rng.choice(["f32", "8bit"]), "tensors": ",".join(map(str, sizes)), "scale": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _sizes(case):
    return [int(v) for v in case["tensors"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    return _prepare_ffn(case, gen) if case["op"] == "ffn" else _prepare_adam(case, gen, int(seed))


def _prepare_ffn(case, gen):
    t, d, f, dt = case["tokens"], case["hidden"], case["inner"], _DT[case["dtype"]]

    def randn(scale, *shape):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dt)

    s = {"case": case}
    # Rows that a norm has left, inside a buffer whose rows are `gap` elements longer.
    s["x"] = randn(1.0, t, d + case["gap"])[:, :d]
    s["wg"], s["wu"] = randn(d ** -0.5, f, d), randn(d ** -0.5, f, d)
    s["wd"] = randn(f ** -0.5, d, f)
    s["residual"] = randn(2.0, t, d) if case["residual"] else None
    if case["dir"] == "step":
        s["dy"] = randn(0.05, t, d)
    if own:
        from dense_convolution_gb300 import head
        s["op"] = head.GatedFeedForward(t, d, f, case["dtype"], case["act"], x_stride=d + case["gap"])
    return s


def _prepare_adam(case, gen, seed):
    sizes = _sizes(case)
    padded = [-(-n // _BLOCK) * _BLOCK for n in sizes]
    total, blocks = sum(padded), sum(padded) // _BLOCK
    s = {"case": case, "sizes": sizes, "seed": 0x9E3779B97F4A7C15 ^ (seed * 0x2545F4914F6CDD1D % 2 ** 64)}
    # One buffer for all weights, as a program keeps it that reduces gradients in one piece; zero between the tensors.
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    at, starts = 0, []
    for n, m in zip(sizes, padded):
        live[at:at + n] = True
        starts.append(at)
        at += m
    s["starts"] = starts
    # Gradients of each block have a size of their own; moments of a run some way in.
    size = torch.pow(10.0, torch.rand(blocks, 1, generator=gen, device="cuda") * 2 - 4)

    def randn(scale):
        x = torch.randn(total, generator=gen, device="cuda").view(blocks, _BLOCK).mul_(scale).view(-1)
        return x.mul_(live)

    s["p"] = randn(0.05)
    s["g"] = randn(size * 1024 if case["grad"] == "f16" and case["scale"] else size).to(_DT[case["grad"]])
    s["copy"] = s["p"].to(_DT[case["copy"]]) if case["copy"] else None
    m = randn(size * 0.3)
    v = (m * m + randn(size * 0.8).square_()).contiguous()
    if case["states"] == "8bit":
        half = torch.full((1,), 1 << 15, dtype=torch.int32, device="cuda")
        s["m"], s["m_scale"] = _to8(m, half, 8, 3)
        s["v"], s["v_scale"] = _to8(v, half, 15, 2)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    # Matrices decay, gains and offsets do not.
    s["decay"] = [0.1 if n > 4096 else 0.0 for n in sizes]
    s["scale"] = torch.full((), 1.0 / 1024 if case["grad"] == "f16" else 0.7, device="cuda") if case["scale"] else None
    s["step"] = 100 + seed % 1000
    if own:
        from dense_convolution_gb300 import head
        s["op"] = head.AdamW(sizes, case["grad"], case["states"], case["copy"] or None, betas=(_B1, _B2), eps=_EPS,
                             weight_decay=s["decay"])
        s["params"] = [s["p"][a:a + n] for a, n in zip(starts, sizes)]
        s["grads"] = [s["g"][a:a + n] for a, n in zip(starts, sizes)]
        s["copies"] = [s["copy"][a:a + n] for a, n in zip(starts, sizes)] if case["copy"] else None
        s["state"] = head.AdamWState(s["m"], s["v"], s["m_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if c["op"] == "ffn":
        return _own_ffn(s, c) if own else _plain_ffn(s, c)
    # The step that this pass makes: in place, as training goes on.
    if own:
        s["op"](s["params"], s["grads"], s["state"], s["step"], _LR, copies=s["copies"], grad_scale=s["scale"],
                seed=s["seed"])
    else:
        _plain_adam(s, c)
    s["step"] += 1
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if c["copy"]:
        out["copy"] = s["copy"]
    if c["states"] == "8bit":
        out["m_scale"], out["v_scale"] = s["m_scale"], s["v_scale"]
    return out


def _own_ffn(s, c):
    op = s["op"]
    if c["dir"] == "fwd":
        return {"y": op(s["x"], s["wg"], s["wu"], s["wd"], residual=s["residual"])}
    y, saved = op(s["x"], s["wg"], s["wu"], s["wd"], residual=s["residual"], save=True)
    dx, dwg, dwu, dwd = op.backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], saved)
    return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}


# ------------------------------------------------------------------ plain forms (32 bits)
def _act(kind, g):
    """act(g) and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        phi = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k, c = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(k * (g + c * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * c * g * g)


def _plain_ffn(s, c):
    dt = _DT[c["dtype"]]
    x, wg, wu, wd = s["x"].float(), s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u = x @ wg.T, x @ wu.T
    a, slope = _act(c["act"], g)
    h = a * u
    y = h @ wd.T
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(dt)}
    if c["dir"] == "step":
        dy = s["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * slope, dh * a
        out["dx"] = (dg @ wg + du @ wu).to(dt)
        out["dwg"], out["dwu"], out["dwd"] = (dg.T @ x).to(dt), (du.T @ x).to(dt), (dy.T @ h).to(dt)
    return out


_M = 0xFFFFFFFF


def _words(seed, step, sizes, total):
    """A 32-bit number for each element of the padded tensors, as int64."""
    lengths = torch.tensor(sizes, device="cuda")
    quads = torch.div(lengths + (_BLOCK - 1), _BLOCK, rounding_mode="floor") * (_BLOCK // 4)
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), quads, output_size=total // 4)
    first = torch.cumsum(quads, 0) - quads
    c0, c1 = torch.arange(total // 4, device="cuda") - first[tensor], tensor
    c2, c3 = torch.full_like(c0, step & _M), torch.full_like(c0, step >> 32)
    k0, k1 = seed & _M, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # the low 64 bits, wrapped
        c0, c1, c2, c3 = ((p1 >> 32) & _M) ^ c1 ^ k0, p1 & _M, ((p0 >> 32) & _M) ^ c3 ^ k1, p0 & _M
        k0, k1 = (k0 + 0x9E3779B9) & _M, (k1 + 0xBB67AE85) & _M
    return torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)


def _to8(x, noise, top, digits):
    """x in 8 bits and its blocks' scales (as e8m0).  noise: 16 bits added below the last kept one;
    top: the exponent of the largest binade; digits: bits of the significand after the leading one."""
    lowest = 1 - {3: 7, 2: 15}[digits]                     # exponent of the smallest normal value
    bits = x.abs().view(torch.int32).view(-1, _BLOCK)
    most = bits.amax(dim=1, keepdim=True)
    exponent = ((most + (1 << 21) - 1) >> 23) - 127        # one more where the largest is above 1.75
    scale = (exponent - top).clamp(min=-127)
    y = x.abs().view(-1, _BLOCK) * ((127 - scale) << 23).view(torch.float32)
    drop = 23 - digits
    noise = noise.view(-1, _BLOCK) if noise.numel() > 1 else noise
    normal = ((y.view(torch.int32) + (noise << (drop - 16))) >> drop) - ((lowest + 126) << digits)
    small = ((y * 2.0 ** (digits - lowest + 16)).clamp(max=2.0 ** 24).to(torch.int32) + noise) >> 16
    code = torch.where(y < 2.0 ** lowest, small, normal)
    if digits == 2:                                        # v: above zero stays above zero
        code = torch.where(y > 0, code.clamp(min=1), code)
    code = code.to(torch.uint8).view(-1) | torch.where(x < 0, 128, 0).to(torch.uint8)
    kind = torch.float8_e4m3fn if digits == 3 else torch.float8_e5m2
    return code.view(kind), (scale + 127).to(torch.uint8).view(-1).view(torch.float8_e8m0fnu)


def _from8(x, scale):
    byte = scale.view(torch.uint8).to(torch.int32)
    factor = torch.where(byte > 0, byte << 23, 1 << 22).view(torch.float32)     # 2^-127 is no normal value
    return (x.float().view(-1, _BLOCK) * factor[:, None]).view(-1)


def _plain_adam(s, c):
    sizes, t, total = s["sizes"], s["step"], s["p"].numel()
    eight = c["states"] == "8bit"
    g = s["g"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    m = _from8(s["m"], s["m_scale"]) if eight else s["m"]
    v = _from8(s["v"], s["v_scale"]) if eight else s["v"]
    m = _B1 * m + (1.0 - _B1) * g
    v = _B2 * v + (1.0 - _B2) * g * g
    lengths = torch.tensor(sizes, device="cuda")
    blocks = torch.div(lengths + (_BLOCK - 1), _BLOCK, rounding_mode="floor")
    shrink = torch.repeat_interleave(torch.tensor([1.0 - _LR * d for d in s["decay"]], device="cuda"), blocks,
                                     output_size=total // _BLOCK)
    p = (s["p"].view(-1, _BLOCK) * shrink[:, None]).view(-1)
    p = p - _LR / (1.0 - _B1 ** t) * (m / (torch.sqrt(v) * (1.0 - _B2 ** t) ** -0.5 + _EPS))
    s["p"].copy_(p)
    if c["copy"]:
        s["copy"].copy_(p)
    if eight:
        words = _words(s["seed"], t, sizes, total)
        for name, x, noise, top, digits in (("m", m, words & 0xFFFF, 8, 3), ("v", v, words >> 16, 15, 2)):
            code, scale = _to8(x, noise.to(torch.int32), top, digits)
            s[name].view(torch.uint8).copy_(code.view(torch.uint8))
            s[name + "_scale"].view(torch.uint8).copy_(scale.view(torch.uint8))
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "adam":
        return _exact_adam(s, case)
    # Nine products of 2 tokens hidden inner operations at about 1 TFLOP/s.
    if case["tokens"] * case["hidden"] * case["inner"] * (18 if case["dir"] == "step" else 6) > 1.4e13:
        return None
    return _exact_ffn(s, case)


def _exact_ffn(s, c):
    x, wg, wu, wd = (s[k].to(torch.float64) for k in ("x", "wg", "wu", "wd"))
    g = torch.mm(x, wg.t()).requires_grad_(True)
    with torch.enable_grad():
        if c["act"] == "silu":
            a = torch.nn.functional.silu(g)
        else:
            a = torch.nn.functional.gelu(g, approximate="tanh" if c["act"] == "gelu_tanh" else "none")
        slope, = torch.autograd.grad(a.sum(), g)
    a, u = a.detach(), torch.mm(x, wu.t())
    h = a.mul(u)
    y = torch.mm(h, wd.t())
    out = {"y": y if s["residual"] is None else y.add_(s["residual"])}
    if c["dir"] == "step":
        dy = s["dy"].to(torch.float64)
        dh = torch.mm(dy, wd)
        du = dh * a
        dg = dh.mul_(u).mul_(slope)
        out["dx"] = torch.addmm(torch.mm(du, wu), dg, wg)
        out["dwg"], out["dwu"], out["dwd"] = torch.mm(dg.t(), x), torch.mm(du.t(), x), torch.mm(dy.t(), h)
    return out


def _exact_noise(s):
    """The two 16-bit numbers of every element, by numpy, a tensor at a time."""
    low, parts = np.uint64(_M), []
    for k, n in enumerate(s["sizes"]):
        x = np.zeros((4, -(-n // _BLOCK) * (_BLOCK // 4)), dtype=np.uint64)
        x[0] = np.arange(x.shape[1], dtype=np.uint64)
        x[1], x[2], x[3] = k, s["step"] % 2 ** 32, s["step"] // 2 ** 32
        key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
        for r in range(10):
            a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            ka, kb = (np.uint64((key[0] + r * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + r * 0xBB67AE85) % 2 ** 32))
            x = np.stack([(b >> np.uint64(32)) ^ x[1] ^ ka, b & low, (a >> np.uint64(32)) ^ x[3] ^ kb, a & low])
        parts.append(np.ascontiguousarray(x.T.astype("<u4")).view("<u2").reshape(-1, 2))
    return torch.from_numpy(np.concatenate(parts).astype(np.int32)).cuda().double()


def _exact_8(x, noise, top, digits):
    """The 8-bit values of x in 64 bits: on the grid of each value's binade, up with the noise's chance."""
    lowest = 1 - {3: 7, 2: 15}[digits]
    x = x.view(-1, _BLOCK)
    fraction, exponent = torch.frexp(x.abs().amax(dim=1, keepdim=True))     # fraction in [0.5, 1), or zero
    exponent = exponent.double() - 1 + (fraction > 0.875)
    scale = torch.where(fraction > 0, exponent - top, -127.0).clamp(min=-127)
    y = x.abs() * torch.exp2(-scale)
    binade = (torch.frexp(y)[1].double() - 1).clamp(min=lowest)
    grid = torch.exp2(binade - digits)
    code = torch.floor(y / grid + noise.view(-1, _BLOCK) / 65536.0) * grid
    if digits == 2:
        code = torch.where((y > 0) & (code == 0), 2.0 ** (lowest - digits), code)
    return (code * torch.sign(x)).view(-1), torch.exp2(scale).view(-1)


def _exact_adam(s, c):
    t, eight = s["step"], c["states"] == "8bit"
    g = s["g"].double()
    if s["scale"] is not None:
        g *= s["scale"].double()

    def moment(k):
        x = s[k].double()
        return (x.view(-1, _BLOCK) * s[k + "_scale"].double()[:, None]).view(-1) if eight else x

    m = torch.lerp(g, moment("m"), _B1)
    v = torch.lerp(g * g, moment("v"), _B2)
    p = s["p"].double()
    update = (m / (1 - _B1 ** t)) / ((v / (1 - _B2 ** t)).sqrt() + _EPS)
    for start, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        update[start:start + n] += decay * p[start:start + n]
    p -= _LR * update
    out = {"p": p, "m": m, "v": v}
    if c["copy"]:
        out["copy"] = p
    if eight and s["p"].numel() > 3e7:                     # the host's random numbers take too long
        out["m"] = out["v"] = out["m_scale"] = out["v_scale"] = None
    elif eight:
        noise = _exact_noise(s)
        out["m"], out["m_scale"] = _exact_8(m, noise[:, 0], 8, 3)
        out["v"], out["v_scale"] = _exact_8(v, noise[:, 1], 15, 2)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "": 0}
    if case["op"] == "adam":
        n = sum(_sizes(case))
        # p, m and v read and written, g read, the copy written.
        states = 4 * n + 4 * (n // _BLOCK) if case["states"] == "8bit" else 16 * n
        return {"bytes": 8 * n + size[case["grad"]] * n + size[case["copy"]] * n + states, "flops": 15 * n}
    t, d, f, e = case["tokens"], case["hidden"], case["inner"], size[case["dtype"]]
    rows = 3 if case["residual"] else 2
    if case["dir"] == "fwd":
        return {"bytes": (rows * t * d + 3 * d * f) * e, "flops": 6 * t * d * f}
    return {"bytes": ((rows + 2) * t * d + 6 * d * f) * e, "flops": 18 * t * d * f}
