"""AdamW where second moments and eps leave the usual range.

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
