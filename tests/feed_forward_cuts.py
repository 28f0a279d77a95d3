"""Which kernel a feed-forward call takes by its sizes and the number of multiprocessors, restated
from the rules, and cases that take every one of them."""
from __future__ import annotations

import random


def up(a, b):
    return -(-a // b)


def shared_out(small, stages, sms, most=8):
    """CTAs that share a tile of 128 x 128, and the stages one goes through."""
    split, least = 1, up(small, sms) * stages
    for s in (2, 3, 4, 6, 8):
        if s <= most and s * small <= (sms * 7 // 8 if s > 2 else sms) and up(stages, s) + 8 < least:
            split, least = s, up(stages, s) + 8
    return split, least


def tiles(m, n, size):
    return up(m, size) * up(n, size)


def cut(m, n, outputs, stages, sms, most):
    split, least = shared_out(tiles(m, n, 128) * outputs, stages, sms, most)
    wide = up(tiles(m, n, 256) * outputs, sms // 2) * stages
    return "tiles 256x256 split=1" if wide < least else f"tiles 128x128 split={split}"


def matmul(m, n, k, lines, sms):
    if m <= 16 or (m <= 32 and n * k <= 6 << 20):
        return f"scale_lines={lines} tokens={8 if m <= 8 else 16 if m <= 16 else 32} " \
               f"warps={8 if up(n, 16) <= 2 * sms else 4}"
    where = cut(m, n, 1, up(k, 128), sms, 8)
    size, split = where.rsplit(" ", 1)
    return f"scale_lines={lines} {size} rows={64 if m <= 64 and '128x128' in size else 128} {split}"


def matmul_kernels():
    out = {f"scale_lines={ln} tokens={t} warps={w}" for ln in (1, 128) for t in (8, 16, 32) for w in (4, 8)}
    out |= {f"scale_lines={ln} tiles 128x128 rows={r} split={s}" for ln in (1, 128) for r in (64, 128)
            for s in (1, 2, 3, 4, 6, 8)}
    return out | {f"scale_lines={ln} tiles 256x256 rows=128 split=1" for ln in (1, 128)}


def gated(m, d, f, dtype, sms):
    weights = 2 * f * d
    if m <= 8 or (m <= 16 and weights <= 48 << 20) or (m <= 32 and weights <= 8 << 20):
        return {f"gated {dtype} tokens={8 if m <= 8 else 16 if m <= 16 else 32}"}
    return {f"gated {dtype} " + cut(m, 2 * f, 1, up(d, 64), sms, 4)}


def gated_kernels():
    return {f"gated {t} {k}" for t in ("bf16", "f16") for k in (
        "tokens=8", "tokens=16", "tokens=32", "tiles 256x256 split=1",
        *(f"tiles 128x128 split={s}" for s in (1, 2, 3, 4)))}


def backward(m, d, f, dtype, sms):
    if m <= 8:
        few = 1 if m <= 1 else 2 if m <= 2 else 4 if m <= 4 else 8
        return {f"gated gradients {dtype} tokens=8", f"gated dx {dtype} tokens={few}",
                f"gated dw {dtype} tokens={few}"}
    return {f"gated gradients {dtype} " + cut(m, 2 * f, 1, up(d, 64), sms, 4),
            f"gated dx {dtype} " + cut(m, d, 1, 2 * up(f, 64), sms, 8),
            f"gated dw {dtype} " + cut(f, d, 2, up(m, 64), sms, 8)}


def backward_kernels():
    out = set()
    for t in ("bf16", "f16"):
        out |= {f"gated gradients {t} {k}" for k in (
            "tokens=8", "tiles 256x256 split=1", *(f"tiles 128x128 split={s}" for s in (1, 2, 3, 4)))}
        for what in ("dx", "dw"):
            out |= {f"gated {what} {t} {k}" for k in (
                *(f"tokens={n}" for n in (1, 2, 4, 8)), "tiles 256x256 split=1",
                *(f"tiles 128x128 split={s}" for s in (1, 2, 3, 4, 6, 8)))}
    return out


def cases(kernels, draw, most_work):
    """Cheap cases that take all of `kernels`: `draw(rng)` gives (case, what it takes, its work)."""
    rng, left, found = random.Random(1), set(kernels), []
    pool = sorted((c for c in (draw(rng) for _ in range(60000)) if c[2] <= most_work), key=lambda c: c[2])
    for case, takes, _ in pool:
        if takes & left:
            left -= takes
            found.append((case, takes))
    return found, left


def size(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def matmul_cases(sms):
    def draw(rng):
        m = size(rng, 1, 600)
        n, k, lines = size(rng, 40, 12000), size(rng, 100, 6000), rng.choice((1, 128))
        return (m, n, k, lines, rng.choice(("f32", "bf16", "f16"))), {matmul(m, n, k, lines, sms)}, m * n * k
    return cases(matmul_kernels(), draw, 1.5e9)


def gated_cases(sms):
    def draw(rng):
        m, d, f = size(rng, 1, 1500), size(rng, 60, 3000), size(rng, 60, 6000)
        t = rng.choice(("bf16", "f16"))
        return (m, d, f, t, rng.choice(("silu", "gelu", "relu"))), gated(m, d, f, t, sms), m * d * f
    return cases(gated_kernels(), draw, 1.5e9)


def backward_cases(sms):
    def draw(rng):
        m = size(rng, 1, 2500)
        d, f = size(rng, 60, 3000), size(rng, 60, 3000)
        t = rng.choice(("bf16", "f16"))
        return (m, d, f, t, rng.choice(("silu", "gelu", "relu"))), backward(m, d, f, t, sms), m * d * f
    return cases(backward_kernels(), draw, 2.5e9)
