"""What each rounding of attention leaves in its output, in the root mean square over a call.

A rounding to nearest at half step h (relative to 1) of a number with mantissa 1 <= m < 2 is off by at most h / m of
it, h / (m sqrt(3)) in the root mean square of a uniform spread; over mantissas spread evenly on their
logarithm the mean of 1 / m^2 is (1 - 1/4) / (2 log 2).  A rounding dq of the query moves the output by
scale M dq, M = sum_j w_j (V_j - O) K_j^T, and roundings d_j of p, which is summed before them, by
sum_j w_j V_j d_j.
"""
from __future__ import annotations

import math

import torch

from cache_plain import HALF_ULP, turned

SPREAD = math.sqrt((1 - 0.25) / (2 * math.log(2)) / 3)


def cut(x, bits=11):
    """x rounded to nearest with `bits` bits of mantissa (float16's 11) and any exponent."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)


def attend(pr, q, rotate, of_q=lambda x: x, of_p=lambda x: x):
    """(out, of_q, of_p) in 64 bits, causal, with `of_q` applied to the rotated queries and `of_p` to p: the output
    (tokens, q_heads, dim) and the squared 2-norms that roundings of relative size 1 leave, a row each."""
    group, scale = q.shape[1] // pr.heads, pr.dim ** -0.5
    out = torch.zeros(q.shape, dtype=torch.float64)
    parts = torch.zeros(2, *q.shape[:2], dtype=torch.float64)
    starts, qr = pr.starts.cpu().tolist(), of_q(turned(q.cpu(), rotate))
    for b, first in enumerate(starts[:-1]):
        (k, _), (v, _) = pr.held("k", b), pr.held("v", b)
        new, length = starts[b + 1] - first, k.shape[0]
        hidden = torch.arange(length) > length - new + torch.arange(new)[:, None]
        for g in range(q.shape[1]):
            kk, vv, x = k[:, g // group], v[:, g // group], qr[first:first + new, g]
            s = (x @ kk.T * scale).masked_fill(hidden, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            w = p / p.sum(-1, keepdim=True)
            o = of_p(p) @ vv / p.sum(-1, keepdim=True)
            m = torch.einsum("tj,tjd,je->tde", w, vv[None] - o[:, None], kk) * scale
            parts[0, first:first + new, g] = ((m * x[:, None]) ** 2).sum((1, 2))
            parts[1, first:first + new, g] = w ** 2 @ (vv ** 2).sum(-1)
            out[first:first + new, g] = turned(o, rotate)
    return out, parts[0], parts[1]


def ratio(got, pr, q, rotate, dtype, with_q, with_p):
    """The root mean square, over rows, of the error of `got` in parts of that of the roundings: the output's own,
    and of float16 queries and p where `with_q` and `with_p` say so."""
    want, of_q, of_p = attend(pr, q, rotate)
    mean = (HALF_ULP[dtype] * want) ** 2
    mean = mean.sum(-1) + 2.0 ** -22 * (with_q * of_q + with_p * of_p)
    off = ((got.double().cpu() - want) ** 2).sum(-1)
    return math.sqrt((off / mean).mean()) / SPREAD


# (news, lens, heads, group, dim): rows of 8 and 16 for each key head, and many
FEW = [([1] * 10, [150 + 31 * i for i in range(10)], 2, 8, 64), ([1] * 10, [150 + 31 * i for i in range(10)], 2, 8, 128),
       ([4] * 4, [200, 333, 150, 500], 2, 4, 64), ([4] * 4, [200, 333, 150, 500], 2, 4, 128)]
MANY = [([40, 90], [300, 190], 2, 2, 64), ([40, 90], [300, 190], 2, 2, 128)]
# Sizes of queries: scores that lie close, where roundings of p count, and far apart, where those of queries do.
SIZES = (0.1, 0.4)
MOST = 1.2  # of `ratio`: spreads are not quite even, and some thousand numbers have a mean of their own


def problem(shape, size, dtype, device, seed=41):
    from cache_plain import REALS, Problem
    news, lens, heads, group, dim = shape
    torch.manual_seed(seed)
    pr = Problem(news, lens, heads, dim, 16, seed=seed, device=device)
    return pr, (torch.randn(pr.tokens, heads * group, dim) * size).to(REALS[dtype]).to(device)
