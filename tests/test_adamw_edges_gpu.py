"""AdamW where second moments and eps leave the usual range, and 8-bit moments of long tensors, whose
blocks a warp takes in turn.

Bounds of p are test_adamw_gpu's: 16 e of the update with e = 2^-24, m's and v's own errors, 5 e of p.  A second moment
below the smallest normal number, 2^-126, keeps fewer digits: it is off by up to 2^-149 (rounding to nearest, twice), its
root relatively by half of that."""
import numpy as np
import pytest

from .test_adamw_gpu import E, Problem, _codes, _lib, _values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-8, 1e-20, 1e-30, 2.0 ** -126])
@pytest.mark.parametrize("beta2", [0.0, 0.95])
@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_vanishing_second_moments(states, beta2, eps):
    """v from 2^-149 to 2^-100, under an eps that does not hide its root."""
    import torch
    from dense_convolution_gb300 import head
    n, b1 = 50, 0.9
    op = head.AdamW([n], "f32", states, betas=(b1, beta2), eps=eps)
    p = torch.zeros(n, device="cuda")
    g = torch.exp2(torch.arange(-74.0, -74.0 + n / 2, 0.5, device="cuda")) * torch.tensor([1.0, -1.5], device="cuda").repeat(n // 2)
    lr = 2.0 ** -10
    op([p], [g], op.new_state(), 1, lr)
    a2 = float(np.float32(1 - beta2))
    m, v = (1 - b1) * g.double(), a2 * g.double() ** 2
    v_off = 8 * E * v + 2 * 2.0 ** -149
    den = v.sqrt() / (1 - beta2) ** 0.5 + eps
    # The root of v - v_off and of v + v_off, on either side.
    low, high = ((v + s * v_off).clamp(min=0).sqrt() / (1 - beta2) ** 0.5 + eps for s in (-1, 1))
    rate = lr / (1 - b1)
    want = -rate * m / den
    off = rate * (m.abs() * (1 / low - 1 / high) + 4 * E * m.abs() / low) + 16 * E * want.abs() + 1e-44
    assert ((p.double() - want).abs() <= off).all(), ((p.double() - want).abs() / off).tolist()


def test_blocks_of_widely_different_second_moments():
    """v above zero is never stored as zero, however far below the block's largest one it is."""
    import torch
    from dense_convolution_gb300 import head
    op = head.AdamW([512], "f32", "8bit", betas=(0.9, 0.95))
    p, g = torch.zeros(512, device="cuda"), torch.full((512,), 1e-21, device="cuda")
    g[100], g[300] = 1e15, 0.0
    state = op.new_state()
    op([p], [g], state, 1, 1e-3)
    codes = state.v.view(torch.uint8)
    live = g != 0
    assert (codes[live] > 0).all() and codes[300] == 0


def _words(seed, step, tensor, n):
    """The 32-bit number of each of the first n elements of a tensor, on the GPU as int64."""
    import torch
    low = 0xffffffff
    c0 = torch.arange(-(-n // 4), device="cuda")
    c1, c2, c3 = (torch.full_like(c0, k) for k in (tensor, step & low, step >> 32))
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32) & low ^ c1 ^ k0, b & low, (a >> 32) & low ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1).view(-1)[:n]


def _expected(q, t, seed, before):
    """Codes and scales of every tensor after step t, by test_adamw_gpu's rule on the host."""
    import torch
    m0, v0 = before
    for i, n in enumerate(q.sizes):
        pad = -n % 256
        host = lambda x: np.pad(x.float().cpu().numpy(), (0, pad))
        s = slice(q.at[i], q.at[i] + n)
        g = host(q.g[i])
        m = np.float32(0.9) * host(m0[s]) + np.float32(1 - 0.9) * g
        v = np.float32(0.95) * host(v0[s]) + np.float32(1 - 0.95) * g * g
        w = _words(seed, t, i, n + pad).cpu().numpy()
        yield i, n + pad, _codes(m, w & 0xffff, "m"), _codes(v, w >> 16, "v")


@pytest.mark.parametrize("grad,copy,shift", [("bf16", "bf16", 0), ("f32", None, 0), ("f16", "f16", 0), ("bf16", "f16", 1)])
def test_long_8bit_tensors(grad, copy, shift):
    """Above 2^24 elements a warp takes eight blocks in turn, the next two on their way: tensors that end inside that,
    in a ragged block, in the first one, or whose addresses fit no vector have the codes of the rule."""
    import torch
    sizes = [(1 << 23) + 8 * 1024 + 3 * 1024 + 5 * 256 + 77, 700, (1 << 22) + 256 * 4, 0, 256, 5 * 1024 + 1, (1 << 22) + 8191, 1 << 20]
    q = Problem(sizes, grad, "8bit", copy, shift, seed=31)
    assert q.op.elements >= 1 << 24
    for t in (1, 2, 3):
        ps, (m0, v0) = [p.clone() for p in q.p], q.moments()
        q.step(t, seed=77)
        for i, n, m, v in _expected(q, t, 77, (m0, v0)):
            whole = slice(q.at[i], q.at[i] + n)
            blocks = slice(whole.start // 256, whole.stop // 256)
            for kind, (codes, scales) in (("m", m), ("v", v)):
                assert np.array_equal(getattr(q.state, kind).view(torch.uint8)[whole].cpu().numpy(), codes), (t, i, kind)
                assert np.array_equal(getattr(q.state, kind + "_scale").view(torch.uint8)[blocks].cpu().numpy(), scales), (t, i, kind)
        for i, n in enumerate(sizes):
            s = slice(q.at[i], q.at[i] + n)
            g = q.g[i].double()
            m, v = 0.9 * m0[s].double() + (1 - 0.9) * g, 0.95 * v0[s].double() + (1 - 0.95) * g * g
            den, rate = v.sqrt() / (1 - 0.95 ** t) ** 0.5 + 1e-8, 1e-2 / (1 - 0.9 ** t)
            want = ps[i].double() * (1 - 1e-2 * q.decay[i]) - rate * m / den
            m_off = 4 * E * (0.9 * m0[s].double().abs() + (1 - 0.9) * g.abs()) + 1e-44
            off = 5 * E * ps[i].double().abs() + rate * (m_off + 16 * E * m.abs()) / den + 1e-44
            assert ((q.p[i].double() - want).abs() <= off).all(), (t, i)
            if copy:
                assert q.c[i].equal(q.p[i].to(q.c[i].dtype)), (t, i)
    for buf, at, n in q.buffers:
        assert torch.isnan(buf[:at]).all() and torch.isnan(buf[at + n:]).all() and not torch.isnan(buf[at:at + n]).any()


def test_a_tensor_given_twice_is_refused():
    import torch
    from dense_convolution_gb300 import head
    op = head.AdamW([64, 64, 0, 0], "bf16", "f32", "bf16")
    z = lambda n, dtype=torch.bfloat16: torch.zeros(n, dtype=dtype, device="cuda")
    p, g, c = [z(64, torch.float32), z(64, torch.float32), z(0, torch.float32), z(0, torch.float32)], [z(64), z(64), z(0), z(0)], [z(64), z(64), z(0), z(0)]
    state = op.new_state()
    op(p, [g[0], g[0], g[2], g[2]], state, 1, 0.1, copies=c)       # a gradient is only read
    for params, copies in ((p, [c[0], c[0], c[2], c[3]]), ([p[1], p[1], p[2], p[3]], c)):
        with pytest.raises(ValueError):
            op(params, g, state, 1, 0.1, copies=copies)
