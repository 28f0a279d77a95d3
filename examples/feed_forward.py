"""A feed-forward block whose down projection runs in 8 bits, trained and served.

    y = (act(x Wg^T) * (x Wu^T)) Wd^T

The gated projections and their gradients run in bfloat16; the down projection and both of
its gradient products in 8 bits with a scale for each block of 128, every operand rotated
along the contraction before it is quantised.

    python examples/feed_forward.py [--steps N] [--tokens M] [--width D] [--hidden F]

trains the block towards a fixed random one, then feeds the same tokens one at a time, as a
decoder would, and prints how far the two ways are apart.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import walsh_hadamard_transform_gb300 as fwt  # noqa: E402

ROTATE = 7  # groups of 128: as far as one scale reaches


class FeedForward:
    """Weights in float32, with their working copies laid out once a step."""

    def __init__(self, width, hidden, seed, activation="silu"):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda rows, cols: torch.randn(rows, cols, device="cuda", generator=gen) * cols ** -0.5  # noqa: E731
        self.weights = {"gate": make(hidden, width), "up": make(hidden, width),
                        "down": make(width, hidden)}
        self.activation = activation
        self.lay_out()

    def lay_out(self):
        self.gate, self.up, down = (self.weights[n].bfloat16() for n in ("gate", "up", "down"))
        # Wd along its rows for y = h Wd^T, and along its columns for dh = dy Wd
        self.down = fwt.quantize_blocks(down, rotate=ROTATE, lines=128)
        self.down_t = fwt.quantize_blocks(down, rotate=ROTATE, axis=0, lines=128)

    def forward(self, x):
        """y, and what the backward pass needs."""
        h = fwt.gated(x, self.gate, self.up, activation=self.activation)
        y = fwt.matmul_blocks(*fwt.quantize_blocks(h, rotate=ROTATE), *self.down)
        return y, (x, h)

    def backward(self, dy, saved):
        """Gradients of the weights and of x."""
        x, h = saved
        # dh = dy Wd runs along the width; dWd = dy^T h along the tokens, so both of its
        # operands are quantised down the rows
        dh = fwt.matmul_blocks(*fwt.quantize_blocks(dy, rotate=ROTATE), *self.down_t)
        d_down = fwt.matmul_blocks(*fwt.quantize_blocks(dy, rotate=ROTATE, axis=0),
                                   *fwt.quantize_blocks(h, rotate=ROTATE, axis=0),
                                   out_dtype=torch.float32)
        dx, d_gate, d_up = fwt.gated_backward(dh, x, self.gate, self.up, activation=self.activation)
        return {"gate": d_gate, "up": d_up, "down": d_down}, dx

    def step(self, gradients, rate):
        for name, g in gradients.items():
            self.weights[name] -= rate * g.float()
        self.lay_out()


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=30)
    parser.add_argument("--tokens", type=int, default=512)
    parser.add_argument("--width", type=int, default=512)
    parser.add_argument("--hidden", type=int, default=1408)
    args = parser.parse_args(argv)

    teacher = FeedForward(args.width, args.hidden, seed=1)
    student = FeedForward(args.width, args.hidden, seed=2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(args.tokens, args.width, device="cuda", generator=gen).bfloat16()
    target, _ = teacher.forward(x)
    losses = []
    for step in range(args.steps):
        y, saved = student.forward(x)
        error = y.float() - target.float()
        losses.append(error.square().mean().item())
        gradients, _ = student.backward((error * (2 / args.tokens)).bfloat16(), saved)
        student.step(gradients, rate=0.05)
        if step % 10 == 0:
            print(f"step {step}: loss {losses[-1]:.5f}")
    print(f"step {args.steps}: loss {losses[-1]:.5f}")

    together, _ = student.forward(x[:16])
    one_by_one = torch.cat([student.forward(x[i:i + 1])[0] for i in range(16)])
    gap = ((one_by_one.float() - together.float()).norm() / together.float().norm()).item()
    print(f"one token at a time against a batch: relative difference {gap:.2e}")
    return losses, gap


if __name__ == "__main__":
    main()
