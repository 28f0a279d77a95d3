"""The feed-forward operators together: the example's block, its gradients and its two ways
of serving, against 64 bits."""
import os
import sys

import pytest
import torch

import feed_forward_plain as plain

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_block_and_its_gradients():
    """One forward and backward pass.  e4m3 keeps 4 significant bits: each operand of the 8-bit
    products is off by at most 2^-4, uniformly within a step, so by at most 2^-4 / sqrt(3) in
    the 2-norm; the products add the errors of their two operands, the others' 2^-8 are small
    beside them.  The gradients through dh carry one such product, dWd one with h's own."""
    import feed_forward
    block = feed_forward.FeedForward(256, 648, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(300, 256, device="cuda", generator=gen).bfloat16()
    y, saved = block.forward(x)
    dy = torch.randn(300, 256, device="cuda", generator=gen).bfloat16()
    gradients, dx = block.backward(dy, saved)

    wd = block.weights["down"].bfloat16().double().cpu()
    xd, dyd = x.double().cpu(), dy.double().cpu()
    h = plain.gated(x, block.gate, block.up, "silu")
    dh = dyd @ wd
    want = dict(zip(("x", "gate", "up"), plain.gated_backward(dh, x, block.gate, block.up, "silu")))
    want.update(y=h @ wd.t(), down=dyd.t() @ h)
    got = dict(gradients, x=dx, y=y)
    one = 2.0 ** -4 / 3 ** 0.5
    for name, w in want.items():
        off = ((got[name].double().cpu() - w).norm() / w.norm()).item()
        assert off <= 2 * one + 2.0 ** -7, (name, off)
    assert xd.shape == dx.shape


def test_example_trains_and_serves(capsys):
    import feed_forward
    losses, gap = feed_forward.main(["--steps", "12", "--tokens", "200", "--width", "256",
                                     "--hidden", "520"])
    assert losses[-1] < 0.7 * losses[0] and all(b < a for a, b in zip(losses[:6], losses[1:6]))
    # the same formulas in another order of fp32 sums: h may round to a neighbour in 8 bits
    # of mantissa and its codes with it
    assert gap <= 2.0 ** -6
    assert "one token at a time" in capsys.readouterr().out
