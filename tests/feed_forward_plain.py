"""The feed-forward operators in 64 bits on the host, from their definitions, for the tests."""
from __future__ import annotations

import math

import torch

REALS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a unit in the last place, relative, and the absolute rounding below the normal range
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -149}


def hadamard(r):
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(r):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h * 2.0 ** (-r / 2)


def rotated(x, r, axis):
    """y (lines, L): each group of 2^r along the axis rotated, zero-extended to whole groups."""
    y = x.double().cpu()
    y = y if axis == 1 else y.t()
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % (1 << r)))
    return (y.reshape(-1, 1 << r) @ hadamard(r)).reshape(y.shape)


def block_max(y, lines):
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % 128, 0, -y.shape[0] % lines))
    return y.view(y.shape[0] // lines, lines, y.shape[1] // 128, 128).abs().amax(dim=(1, 3))


def spread(scale, lines, rows, length):
    return (scale.double().cpu().repeat_interleave(lines, 0)[:rows]
            .repeat_interleave(128, 1)[:, :length])


def e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even."""
    exponent = torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 1
    step = 2.0 ** (exponent - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def values(q):
    return q.cpu().float().double()


def activation(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 0.134145 * g * g)
    return g.clamp(min=0), (g > 0).double()


def gated(x, wg, wu, act):
    x, wg, wu = (t.double().cpu() for t in (x, wg, wu))
    return activation(x @ wg.t(), act)[0] * (x @ wu.t())


def gated_parts(grad, x, wg, wu, act):
    grad, x, wg, wu = (t.double().cpu() for t in (grad, x, wg, wu))
    g, u = x @ wg.t(), x @ wu.t()
    value, slope = activation(g, act)
    return grad * u * slope, grad * value


def gated_backward(grad, x, wg, wu, act):
    dg, du = gated_parts(grad, x, wg, wu, act)
    x, wg, wu = (t.double().cpu() for t in (x, wg, wu))
    return dg @ wg + du @ wu, dg.t() @ x, du.t() @ x
