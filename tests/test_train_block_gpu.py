"""The example that trains norm, feed-forward block, dropout and loss with AdamW: it runs
and repeats itself bit for bit, its gradients are those of the same head in 64 bits,
and a captured step is the eager one."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build
    build.build()


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_runs_repeat(states):
    from examples import train_block
    a = train_block.train(steps=6, images=2, vocab=300, states=states, log=None)
    b = train_block.train(steps=6, images=2, vocab=300, states=states, log=None)
    assert a == b and all(math.isfinite(v) for v in a)


def _problem():
    import torch
    from examples import train_block
    g = torch.Generator(device="cuda").manual_seed(7)
    images, channels, pixels, inner, vocab = 3, 96, 100, 200, 500
    head = train_block.Head(images, channels, pixels, inner, vocab, p=0.0, states="8bit")
    head.matrices[3].mul_(10)                               # a head that already has an opinion
    head.copies[3].copy_(head.matrices[3])
    x = torch.randn(images, channels, pixels, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, vocab, (images * pixels,), generator=g, device="cuda")
    target[::9] = train_block.IGNORE
    return head, x, target


def test_gradients():
    """Along the chain three to six roundings to bf16 (2^-8 at most, 0.43 of that in the mean) add up as
    their squares: 6^(1/2) 0.43 2^-8 = 4.1e-3 in the 2-norm, and twice that is allowed."""
    import torch
    head, x, target = _problem()
    loss, vectors, matrices = head.gradients(x, target)
    t = [v.double().requires_grad_() for v in head.vectors + head.copies]
    gamma, beta, wg, wu, wd, w = t
    rows = x.double().transpose(1, 2).reshape(-1, x.shape[1])
    m = rows.mean(1, keepdim=True)
    n = (rows - m) / ((rows - m).square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
    g = n @ wg.T
    h = n + ((g / (1 + torch.exp(-g))) * (n @ wu.T)) @ wd.T
    live = target >= 0
    z = (h @ w.T)[live]
    want = (torch.logsumexp(z, 1) - z[torch.arange(len(z)), target[live]]).mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 8.2e-3 * abs(float(want.detach()))
    for k, (a, b) in enumerate(zip(vectors + matrices, t)):
        off = float((a.double() - b.grad).norm() / b.grad.norm())
        assert off < 8.2e-3, (k, off)


def test_a_captured_step_is_the_eager_one():
    import torch
    (a, x, target), (b, _, _) = _problem(), _problem()
    rate = torch.full((), 1e-3, device="cuda")
    a.update(*a.gradients(x, target)[1:], rate)             # (a first pass outside, as graphs want it)
    b.update(*b.gradients(x, target)[1:], rate)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, vectors, matrices = a.gradients(x, target)
        a.update(vectors, matrices, rate)
    for k in range(3):
        rate.fill_(1e-3 * (k + 1))
        graph.replay()
        want, *grads = b.gradients(x, target)
        b.update(*grads, rate)
        assert loss.equal(want)
    assert all(p.equal(q) for p, q in zip(a.vectors + a.matrices + a.copies, b.vectors + b.matrices + b.copies))
    assert all(p.view(torch.uint8).equal(q.view(torch.uint8)) for p, q in zip(a.state[1], b.state[1]))
    assert int(a.step) == int(b.step) == 4
