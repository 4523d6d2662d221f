"""Train a vocabulary head on a frozen convolution layer.

    python examples/train_head.py [--steps 40] [--images 8] [--vocab 2000]

The trunk is one convolution of this library (3x3, NCHW, bf16) with fixed random
filters.  Each output pixel is a token: layer norm turns the feature planes into
token rows, dropout regularises them, and the linear cross entropy scores every
token against the vocabulary.  The gradients come back through the head: dw from
the loss, dgamma and dbeta through dropout and layer norm (the trunk is frozen,
so dx is not asked for).  Targets are what a hidden random head would say, with
a tenth of the tokens ignored.  Prints the loss as it falls.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_convolution_gb300 import capi                                            # noqa: E402
from dense_convolution_gb300.conv import Conv2d                                     # noqa: E402
from dense_convolution_gb300.head import Dropout, LayerNorm, LinearCrossEntropy     # noqa: E402

IGNORE = -100


def train(steps=40, images=8, channels=128, side=28, vocab=2000, p=0.1, lr=2.0, seed=1, log=print):
    """Runs `steps` steps and returns the losses (one float a step)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    tokens = images * side * side

    conv = Conv2d(images, 64, side, side, channels, 3, 3, 1, 1, "bf16", "auto")
    filters = conv.pack_filter((randn(channels, 64, 3, 3) / 24).bfloat16())
    conv.set_prepacked(True)
    norm = LayerNorm(tokens, channels, "bf16", "f32", pixels=side * side)
    drop = Dropout(tokens, channels, "bf16", p)
    loss_of = LinearCrossEntropy(tokens, channels, vocab, "bf16", reduction="mean", ignore_index=IGNORE)

    gamma, beta = torch.ones(channels, device="cuda"), torch.zeros(channels, device="cuda")
    master = 0.02 * randn(vocab, channels)                  # fp32 weights; the products read their bf16 copy
    teacher = randn(vocab, channels).bfloat16()
    one = torch.ones((), device="cuda")
    losses = []
    for step in range(steps):
        x = randn(images, 64, side, side).bfloat16()
        features = conv(x, filters)                         # NCHW planes
        rows, mean, rstd = norm(features, gamma, beta, stats=True)
        with torch.no_grad():                               # this step's targets
            target = (rows.float() @ teacher.float().T).argmax(1)
            target[torch.rand(tokens, generator=gen, device="cuda") < 0.1] = IGNORE
        h = drop(rows, seed, offset=step)
        w = master.bfloat16()
        loss, lse = loss_of(h, w, target)
        dh, dw = loss_of.backward(h, w, target, lse, one)
        _, dgamma, dbeta = norm.backward(drop.backward(dh, seed, offset=step), features, gamma, mean, rstd,
                                         need_dx=False)
        master -= lr * dw.float()
        gamma -= 0.1 * lr * dgamma
        beta -= 0.1 * lr * dbeta
        losses.append(loss)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {float(loss):.4f}")
    status = capi.conv2d_device_status(torch.cuda.current_stream().cuda_stream)
    if status:
        raise RuntimeError(f"device status {status}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--images", type=int, default=8)
    ap.add_argument("--vocab", type=int, default=2000)
    a = ap.parse_args()
    train(a.steps, a.images, vocab=a.vocab)
