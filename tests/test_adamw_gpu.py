"""AdamW over many tensors against its definition, through the public entry points.

With e = 2^-24 (fp32's unit roundoff), k the gradient's factor:
  m    b1 and 1 - b1 are rounded, as are k g, the two products and their sum:
       4 e (|b1 m| + |(1 - b1) k g|).
  v    k g and the product that it enters count twice: 8 e (b2 v + (1 - b2) (k g)^2).
  p    lr decay is a product of rounded factors under one fma (3 e), the product with
       p and the last fma round (2 e).  The update is off by m's own error over the
       denominator, and relatively by half of v's (4 e), the root, its factor, the fma
       with eps, the quotient, lr / c1 and their constants: below 16 e; where the
       device holds t, c1 and c2 come from fp32 exponentials (3 e each): 24 e.
  copy one rounding of p as it was stored: exact.
  8 bits: m and v take fp32 operations that round one by one, and their codes are
       integers of the results' bits: numpy's fp32 gives the same codes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BETAS, EPS = (0.9, 0.95), 1e-8
TOP, DIGITS = {"m": 8, "v": 15}, {"m": 3, "v": 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build
    build.build()


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _words(seed, step, tensor, n):
    """The 32-bit number of each of the first n elements of a tensor."""
    x = [np.arange(-(-n // 4), dtype=np.uint64), np.uint64(tensor), np.uint64(step & 0xffffffff), np.uint64(step >> 32)]
    x = [np.broadcast_to(v, x[0].shape) for v in x]
    k0, k1, low = seed & 0xffffffff, seed >> 32, np.uint64(0xffffffff)
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return np.stack(x, 1).reshape(-1)[:n].astype(np.int64)


def _codes(x, noise, kind):
    """8-bit codes and scale bytes of fp32 x (whole blocks), from the rule in words."""
    top, digits = TOP[kind], DIGITS[kind]
    low = -6 if kind == "m" else -14
    x = x.reshape(-1, 256)
    most = np.abs(x).max(1).view(np.int32).astype(np.int64)
    exponent = (most >> 23) - 127 + ((most & 0x7fffff) > 0x600000)
    scale = np.maximum(exponent - top, -127)
    y = np.abs(x) * np.exp2(-scale.astype(np.float64)).astype(np.float32)[:, None]
    bits = y.view(np.int32).astype(np.int64)
    normal = ((bits + (noise.reshape(-1, 256) << (7 - digits))) >> (23 - digits)) - ((low + 126) << digits)
    small = (np.minimum(y.astype(np.float64) * 2.0 ** (digits - low + 16), 2.0 ** 40).astype(np.int64) + noise.reshape(-1, 256)) >> 16
    code = np.where(y < 2.0 ** low, small, normal)
    if kind == "v":
        code = np.where((y > 0) & (code == 0), 1, code)
    return (code | np.where(np.signbit(x), 128, 0)).reshape(-1).astype(np.uint8), (scale + 127).astype(np.uint8)


def _values(codes, scales):
    """fp32 values of 8-bit moments (torch tensors)."""
    import torch
    byte = scales.view(torch.uint8).to(torch.int32)
    factor = torch.where(byte > 0, byte << 23, 1 << 22).view(torch.float32)
    return (codes.float().view(-1, 256) * factor[:, None]).view(-1)


class Problem:
    """Tensors somewhere in buffers of NaN, `shift` elements past an aligned address."""

    def __init__(self, sizes, grad="f32", states="f32", copy=None, shift=0, seed=1, decay=None, scale=None):
        import torch
        from dense_convolution_gb300 import head
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.states, self.copy_dtype, self.grad, self.k = sizes, states, copy, grad, scale
        self.decay = decay if decay is not None else [0.1 * (i % 3) for i in range(len(sizes))]
        self.buffers = []

        def put(values, dtype):
            buf = torch.full((values.numel() + 64 + shift,), float("nan"), dtype=dtype, device="cuda")
            view = buf[32 + shift:32 + shift + values.numel()]
            view.copy_(values)
            self.buffers.append((buf, 32 + shift, values.numel()))
            return view

        randn = lambda n: torch.randn(n, generator=g, device="cuda")
        self.p = [put(randn(n), torch.float32) for n in sizes]
        self.g = [put(randn(n) * 10.0 ** (i % 4 - 3), _dt(grad)) for i, n in enumerate(sizes)]
        self.c = [put(torch.zeros(n, device="cuda"), _dt(copy)) for n in sizes] if copy else None
        self.op = head.AdamW(sizes, grad, states, copy, BETAS, EPS, self.decay)
        self.state = self.op.new_state()
        self.at = [self.op.offset(i) for i in range(len(sizes))]
        self.scale = torch.full((), scale, device="cuda") if scale else None

    def step(self, t, lr=1e-2, seed=7, **more):
        self.op(self.p, self.g, self.state, t, lr, copies=self.c, grad_scale=self.scale, seed=seed, **more)

    def moments(self):
        if self.states == "f32":
            return self.state.m.clone(), self.state.v.clone()
        return _values(self.state.m, self.state.m_scale), _values(self.state.v, self.state.v_scale)

    def check(self, t, before, lr=1e-2, seed=7, device=False):
        """The state against a step from `before` (p's clones, m, v)."""
        import torch
        b1, b2 = BETAS
        ps, m0, v0 = before
        m1, v1 = self.moments()
        for i, n in enumerate(self.sizes):
            s = slice(self.at[i], self.at[i] + n)
            g = self.g[i].double() * (float(np.float32(self.k)) if self.k else 1.0)
            m, v = b1 * m0[s].double() + (1 - b1) * g, b2 * v0[s].double() + (1 - b2) * g * g
            m_off = 4 * E * (b1 * m0[s].double().abs() + (1 - b1) * g.abs()) + 1e-44
            v_off = 8 * E * v + 1e-44
            if self.states == "f32":
                assert ((m1[s].double() - m).abs() <= m_off).all() and ((v1[s].double() - v).abs() <= v_off).all(), i
            else:
                pad = -n % 256
                f = lambda x: np.pad(x.float().cpu().numpy(), (0, pad))
                k = np.float32(self.k) if self.k else np.float32(1)
                gf = f(self.g[i]) * k
                mf = np.float32(b1) * f(m0[s]) + np.float32(1 - b1) * gf
                vf = np.float32(b2) * f(v0[s]) + np.float32(1 - b2) * gf * gf
                w = _words(seed, t, i, n + pad)
                for kind, x, noise in (("m", mf, w & 0xffff), ("v", vf, w >> 16)):
                    codes, scales = _codes(x, noise, kind)
                    whole = slice(self.at[i], self.at[i] + n + pad)
                    blocks = slice(whole.start // 256, whole.stop // 256)
                    assert np.array_equal(getattr(self.state, kind).view(torch.uint8)[whole].cpu().numpy(), codes), (i, kind)
                    assert np.array_equal(getattr(self.state, kind + "_scale").view(torch.uint8)[blocks].cpu().numpy(), scales), (i, kind)
            den = v.sqrt() / (1 - b2 ** t) ** 0.5 + EPS
            rate = lr / (1 - b1 ** t)
            want = ps[i].double() * (1 - lr * self.decay[i]) - rate * m / den
            off = 5 * E * ps[i].double().abs() + rate * (m_off + (24 if device else 16) * E * m.abs()) / den + 1e-44
            assert ((self.p[i].double() - want).abs() <= off).all(), (i, float(((self.p[i].double() - want).abs() / off).max()))
            if self.c:
                assert self.c[i].equal(self.p[i].to(self.c[i].dtype)), i
        for buf, at, n in self.buffers:                        # what lies beside the tensors stays
            assert torch.isnan(buf[:at]).all() and torch.isnan(buf[at + n:]).all() and not torch.isnan(buf[at:at + n]).any()

    def before(self):
        return ([p.clone() for p in self.p],) + self.moments()


SIZES = [1, 0, 3, 255, 256, 257, 2047, 2048, 2049, 10000, 8, 70000]


@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("grad,copy,shift,scale", [("f32", None, 0, None), ("bf16", "bf16", 0, 0.37), ("f16", "f16", 0, None),
                                                   ("f32", "bf16", 1, 3.0), ("bf16", "f16", 4, None), ("f16", None, 7, 0.001)])
def test_steps(states, grad, copy, shift, scale):
    q = Problem(SIZES, grad, states, copy, shift, seed=shift + 3, scale=scale)
    for t in (1, 2, 3, 1000, (1 << 33) + 5):
        was = q.before()
        q.step(t)
        q.check(t, was)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_more_tensors_than_a_launch_takes(states):
    q = Problem([(i * 37) % 600 for i in range(1500)], "bf16", states, "bf16")
    was = q.before()
    q.step(1)
    q.check(1, was)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_step_and_rate_on_the_device_captured_and_replayed(states):
    import torch
    a, b = (Problem([300, 5000, 64], "f32", states, "f16", seed=9) for _ in range(2))
    t, lr = torch.zeros((), dtype=torch.int64, device="cuda"), torch.full((), 0.02, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            t.add_(1)
            a.step(t, lr)
    torch.cuda.current_stream().wait_stream(side)
    for k in range(1, 5):
        was = a.before()
        lr.fill_(0.02 / k)
        graph.replay()
        torch.cuda.synchronize()
        assert int(t) == k
        a.check(k, was, lr=float(np.float32(0.02 / k)), device=True)
        b.step(k, lr=0.02 / k)
    for x, y in zip(a.moments(), b.moments()):                 # the moments do not depend on where t lies
        assert x.equal(y)


def test_two_graphs_share_nothing_but_the_state():
    import torch
    a, b = Problem([5000], "f32", "8bit", seed=4), Problem([5000], "f32", "8bit", seed=4)
    graphs = []
    for t in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.step(t)
        graphs.append(g)
    graphs[0].replay()
    graphs[1].replay()
    b.step(1)
    b.step(2)
    assert all(x.equal(y) for x, y in zip(a.moments(), b.moments())) and a.p[0].equal(b.p[0])


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_skip(states):
    import torch
    q = Problem([700, 40], "f32", states, "bf16")
    q.step(1)
    was, copies = q.before(), [c.clone() for c in q.c]
    for value in (1.0, float("inf"), float("nan"), -2.0):
        q.step(2, skip=torch.full((), value, device="cuda"))
        now = q.before()
        assert all(x.equal(y) for x, y in zip(was[0] + list(was[1:]) + copies, now[0] + list(now[1:]) + q.c))
    q.step(2, skip=torch.zeros((), device="cuda"))
    q.check(2, was)


def test_blocks_that_are_not_finite_and_zero_gradients():
    import torch
    q = Problem([1024], "f32", "8bit")
    q.g[0][300], q.g[0][600] = float("inf"), float("nan")
    q.step(1)
    bad = torch.zeros(1024, dtype=torch.bool, device="cuda")
    bad[[300, 600]] = True
    assert torch.isnan(q.p[0][bad]).all() and torch.isfinite(q.p[0][~bad]).all()
    assert q.state.m_scale.view(torch.uint8).tolist()[1:3] == [255, 255] == q.state.v_scale.view(torch.uint8).tolist()[1:3]
    q.g[0].zero_()
    q.step(2)
    assert torch.isnan(q.p[0][256:768]).all() and torch.isfinite(q.p[0][:256]).all() and torch.isfinite(q.p[0][768:]).all()
    q = Problem([513], "f32", "8bit", decay=[0.0])
    q.g[0].zero_()
    was = q.p[0].clone()
    q.step(1)
    assert q.p[0].equal(was) and not q.moments()[0].any() and not q.moments()[1].any()


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_a_second_moment_that_overflows(states):
    """v is infinite where the gradient's square is: p stays for the step, as m over infinity says.  In 8 bits the
    block's v is not a number from then on, and neither is what p takes from it, though m is finite."""
    import torch
    q = Problem([1024], "f32", states, decay=[0.0])
    q.g[0][300] = 1e25
    was = q.p[0].clone()
    q.step(1)
    assert float(q.p[0][300]) == float(was[300]) and torch.isfinite(q.p[0]).all()
    q.g[0].zero_()
    q.step(2)
    if states == "f32":
        assert torch.isfinite(q.p[0]).all() and float(q.p[0][300]) == float(was[300])
    else:
        assert torch.isnan(q.p[0][256:512]).all() and torch.isfinite(q.p[0][:256]).all() and torch.isfinite(q.p[0][512:]).all()


def test_8bit_moments_move_as_the_formula_on_average():
    """Without gradients v falls by b2 a step; rounding to nearest would leave it.
    A value's own walk spreads by less than a step of its code in each of a few
    binades; the mean over 2^18 values by 2^-9 of that: 2 % holds it many times over."""
    import torch
    from dense_convolution_gb300 import head
    n = 1 << 18
    op = head.AdamW([n], "f32", "8bit", betas=(0.99, 0.999))
    g = torch.Generator(device="cuda").manual_seed(3)
    p, grad = torch.zeros(n, device="cuda"), torch.randn(n, generator=g, device="cuda").abs() + 0.5
    state = op.new_state()
    op([p], [grad], state, 1, 0.0, seed=1)
    m, v = _values(state.m, state.m_scale), _values(state.v, state.v_scale)
    assert abs(float(m.double().mean() / (0.01 * grad.double()).mean()) - 1) < 0.02
    assert abs(float(v.double().mean() / (0.001 * grad.double() ** 2).mean()) - 1) < 0.02
    grad.zero_()
    for t in range(2, 202):
        op([p], [grad], state, t, 0.0, seed=1)
    m2, v2 = _values(state.m, state.m_scale), _values(state.v, state.v_scale)
    assert abs(float(m2.double().mean() / m.double().mean()) / 0.99 ** 200 - 1) < 0.02
    assert abs(float(v2.double().mean() / v.double().mean()) / 0.999 ** 200 - 1) < 0.02


def test_a_tensor_past_32_bit_indexes():
    import torch
    from dense_convolution_gb300 import head
    n = (1 << 31) + 1003
    op = head.AdamW([5, n], "bf16", "8bit", "bf16", BETAS, EPS)
    p, g, c = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    small = [torch.zeros(5, device="cuda"), torch.zeros(5, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, dtype=torch.bfloat16, device="cuda")]
    at = [0, 1 << 30, (1 << 31) + 2, n - 1]
    for i in at:
        g[i] = 0.5
    op([small[0], p], [small[1], g], op.new_state(), 1, 0.25, copies=[small[2], c])
    for i in at:                                               # the first step goes by lr times the gradient's sign
        assert abs(float(p[i]) + 0.25) < 1e-6 and float(c[i]) == -0.25, i
    assert int(torch.count_nonzero(p)) == len(at) == int(torch.count_nonzero(c))


def test_other_stream():
    import torch
    a, b = Problem([5000, 33], "bf16", "8bit", "bf16", seed=6), Problem([5000, 33], "bf16", "8bit", "bf16", seed=6)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.step(1, stream=side)
    side.synchronize()
    b.step(1)
    torch.cuda.synchronize()
    assert all(x.equal(y) for x, y in zip(a.p + list(a.moments()) + a.c, b.p + list(b.moments()) + b.c))


def test_wrong_tensors_are_refused():
    import torch
    from dense_convolution_gb300 import capi, head
    q = Problem([64, 12], "bf16", "8bit", "f16")
    bad = lambda **k: pytest.raises(ValueError, q.op, **{**dict(params=q.p, grads=q.g, state=q.state, step=1, lr=0.1, copies=q.c), **k})
    bad(params=q.p[:1])
    bad(params=[q.p[0], q.p[0][:12]])
    bad(params=[q.p[0].double(), q.p[1]])
    bad(params=[q.p[0].cpu(), q.p[1]])
    bad(params=[torch.zeros(128, device="cuda")[::2], q.p[1]])
    bad(grads=[q.g[0].float(), q.g[1]])
    bad(grads=[q.g[0], q.g[1][:11]])
    bad(copies=None)
    bad(copies=[q.c[0], q.c[1].float()])
    bad(state=head.AdamWState(q.state.v, q.state.m, q.state.m_scale, q.state.v_scale))
    bad(state=q.state._replace(m_scale=None))
    bad(step=torch.ones((), device="cuda"))
    bad(lr=torch.ones((), dtype=torch.float64, device="cuda"))
    bad(grad_scale=2.0)
    bad(skip=torch.zeros((), dtype=torch.int32, device="cuda"))
    with pytest.raises(capi.Conv2dError):
        q.op(q.p, q.g, q.state, 0, 0.1, copies=q.c)
    with pytest.raises(ValueError):
        head.AdamW([4, 5], weight_decay=[0.1])
    with pytest.raises(ValueError):
        head.AdamW([4], copy_dtype="f32")
    two = head.AdamW([64, 64], "bf16")
    with pytest.raises(ValueError):
        two([q.p[0], q.p[0]], [q.g[0], q.g[0]], two.new_state(), 1, 0.1)
