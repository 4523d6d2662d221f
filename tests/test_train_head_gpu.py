"""The example that trains a vocabulary head on convolution features: the loss
starts at the logarithm of the vocabulary and falls, and a run repeats itself
bit for bit (no operator's result depends on the order in which blocks run)."""
import math

import pytest

pytestmark = pytest.mark.gpu


def test_loss_falls_and_runs_repeat():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build
    build.build()
    from examples import train_head
    a = train_head.train(steps=30, images=4, vocab=500, log=None)
    b = train_head.train(steps=30, images=4, vocab=500, log=None)
    assert a == b
    assert abs(a[0] - math.log(500)) < 0.5
    assert a[-1] < a[0] - 1.0 and all(math.isfinite(v) for v in a)
