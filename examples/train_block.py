"""Train a head with a feed-forward block on a frozen convolution layer.

    python examples/train_block.py [--steps 40] [--images 8] [--vocab 2000] [--states 8bit]

The trunk is one convolution of this library (3x3, NCHW, bf16) with fixed random
filters.  Each output pixel is a token: layer norm turns the feature planes into
token rows, a gated feed-forward block adds to them, dropout regularises them, and the
linear cross entropy scores every token against the vocabulary.  The gradients come
back through all four, and AdamW makes the next weights: fp32 ones, and for the
matrices the bf16 copies that the next step's products read.  Its step number and rate
lie on the GPU, as a captured step would read them.  Targets are what a hidden random
head would say, with a tenth of the tokens ignored.  Prints the loss as it goes.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_convolution_gb300 import capi                                                                # noqa: E402
from dense_convolution_gb300.conv import Conv2d                                                         # noqa: E402
from dense_convolution_gb300.head import (AdamW, Dropout, GatedFeedForward, LayerNorm,                  # noqa: E402
                                          LinearCrossEntropy)

IGNORE = -100


class Head:
    """Norm, block, dropout and loss over `images` feature planes of `channels` by `pixels`."""

    def __init__(self, images, channels, pixels, inner, vocab, p=0.1, states="f32", seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
        tokens = images * pixels
        self.norm = LayerNorm(tokens, channels, "bf16", "f32", pixels=pixels)
        self.block = GatedFeedForward(tokens, channels, inner, "bf16", "silu")
        self.drop = Dropout(tokens, channels, "bf16", p)
        self.loss = LinearCrossEntropy(tokens, channels, vocab, "bf16", reduction="mean", ignore_index=IGNORE)
        # What is trained: gain and offset of the norm; the block's matrices and the vocabulary's.
        self.vectors = [torch.ones(channels, device="cuda"), torch.zeros(channels, device="cuda")]
        self.matrices = [randn(inner, channels) * channels ** -0.5, randn(inner, channels) * channels ** -0.5,
                         randn(channels, inner) * 0.3 * inner ** -0.5, 0.02 * randn(vocab, channels)]
        self.copies = [m.bfloat16() for m in self.matrices]
        self.adam = [AdamW([t.numel() for t in self.vectors], "f32"),
                     AdamW([t.numel() for t in self.matrices], "bf16", states, "bf16", weight_decay=0.01)]
        self.state = [a.new_state() for a in self.adam]
        self.step = torch.zeros((), dtype=torch.int64, device="cuda")
        self.one = torch.ones((), device="cuda")
        self.seed = seed

    def gradients(self, features, target, offset=0):
        """The loss, and the gradients of the vectors and of the matrices."""
        (gamma, beta), (wg, wu, wd, w) = self.vectors, self.copies
        rows, mean, rstd = self.norm(features, gamma, beta, stats=True)
        out, saved = self.block(rows, wg, wu, wd, residual=rows, save=True)
        h = self.drop(out, self.seed, offset=offset)
        loss, lse = self.loss(h, w, target)
        dh, dw = self.loss.backward(h, w, target, lse, self.one)
        dout = self.drop.backward(dh, self.seed, offset=offset)
        drows, dwg, dwu, dwd = self.block.backward(dout, rows, wg, wu, wd, saved)
        drows += dout                                       # through the block, and beside it
        _, dgamma, dbeta = self.norm.backward(drows, features, gamma, mean, rstd, need_dx=False)
        return loss, [dgamma, dbeta], [dwg, dwu, dwd, dw]

    def update(self, vectors, matrices, lr):
        self.step += 1
        self.adam[0](self.vectors, vectors, self.state[0], self.step, lr)
        self.adam[1](self.matrices, matrices, self.state[1], self.step, lr, copies=self.copies, seed=self.seed)


def train(steps=40, images=8, channels=128, side=28, inner=352, vocab=2000, p=0.1, lr=3e-3, states="f32", seed=1, log=print):
    """Runs `steps` steps and returns the losses (one float a step)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    conv = Conv2d(images, 64, side, side, channels, 3, 3, 1, 1, "bf16", "auto")
    filters = conv.pack_filter((randn(channels, 64, 3, 3) / 24).bfloat16())
    conv.set_prepacked(True)
    head = Head(images, channels, side * side, inner, vocab, p, states, seed)
    teacher = randn(vocab, channels).bfloat16()
    rate = torch.full((), lr, device="cuda")
    losses = []
    for step in range(steps):
        x = randn(images, 64, side, side).bfloat16()
        features = conv(x, filters)                         # NCHW planes
        with torch.no_grad():                               # this step's targets
            rows = features.float().flatten(2).transpose(1, 2).reshape(-1, channels)
            target = (rows @ teacher.float().T).argmax(1)
            target[torch.rand(target.numel(), generator=gen, device="cuda") < 0.1] = IGNORE
        loss, vectors, matrices = head.gradients(features, target, offset=step)
        head.update(vectors, matrices, rate)
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
    ap.add_argument("--states", choices=["f32", "8bit"], default="8bit")
    a = ap.parse_args()
    train(a.steps, a.images, vocab=a.vocab, states=a.states)
