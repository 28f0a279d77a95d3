"""The cache operators in 64 bits from their definitions, and inputs for their tests."""
from __future__ import annotations

import math

import torch

from feed_forward_plain import HALF_ULP, REALS, TINY, e4m3, hadamard

E4M3_OF = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
NAN_CODES = (0x7f, 0xff)


def turned(x, r):
    """Each aligned group of 2^r along the last dimension by the normalised H."""
    return (x.double().reshape(-1, 1 << r) @ hadamard(r).to(x.device)).reshape(x.shape)


def raw(t):
    return t.view(torch.uint8)


def quantised(x, r):
    """Values of the codes (before the scale), scale bytes and the rotated x, in 64 bits."""
    y = turned(x, r)
    top = y.abs().amax(-1)
    fine = torch.isfinite(top)
    exponent = torch.ceil(torch.log2(torch.where(fine, top, 1.0).clamp(min=2.0 ** -118) / 448)).clamp(min=-126)
    code = e4m3(y * torch.exp2(-exponent)[..., None])
    return (torch.where(fine[..., None], code, 0.0), torch.where(fine, exponent + 127, 255.0).long(), y)


class Problem:
    """Sequences over a cache of random codes; sizes as the operators take them.  `news`, `lens`: of
    each sequence; `tail`: packed rows behind the last one."""

    def __init__(self, news, lens, heads=2, dim=64, page=16, seed=0, tail=0, device="cuda", spare=3,
                 most_pages=None, codes=True):
        import walsh_hadamard_transform_gb300 as fwt
        gen = torch.Generator().manual_seed(seed)
        self.news, self.lens, self.heads, self.dim, self.page = list(news), list(lens), heads, dim, page
        counts = [-(-n // page) for n in lens]
        self.pages = sum(counts) + spare
        order = torch.randperm(self.pages, generator=gen)
        self.table = torch.full((len(lens), most_pages or max(counts + [1])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.starts = torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32)
        self.lengths = torch.tensor(lens, dtype=torch.int32)
        self.tokens = sum(news) + tail
        self.cache = fwt.new_cache(self.pages, page, heads, dim, device=device)
        if codes:  # any finite code, and scales around 1; what no sequence holds is NaN
            for t in (self.cache.k, self.cache.v):
                c = torch.randint(0, 254, t.shape, generator=gen)
                c = c + (c >= 0x7f).long()
                # (small codes more often than large ones, as of normal values)
                keep = torch.rand(t.shape, generator=gen) < 0.3
                raw(t).copy_(torch.where(keep | (c & 0x7f < 0x40), c, c & 0xbf).to(torch.uint8))
            for t in (self.cache.k_scale, self.cache.v_scale):
                raw(t).copy_(torch.randint(120, 125, t.shape, generator=gen).to(torch.uint8))
            held = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(counts[b]):
                    held[self.table[b, j], :min(page, n - j * page)] = True
            for t in self.cache:
                h = held[:, None].expand(-1, heads, -1).to(t.device)
                raw(t)[~h] = 0x7f if t.dim() == 4 else 0xff
        self.table, self.starts, self.lengths = (t.to(device) for t in (self.table, self.starts, self.lengths))

    def places(self):
        return self.cache, self.table, self.starts, self.lengths

    def held(self, name, b):
        """What the cache holds of sequence b (length, heads, dim) in 64 bits, still rotated, and
        which of its tokens have a page."""
        table = self.table[b].cpu().long()
        length = min(max(int(self.lengths[b]), 0), table.numel() * self.page)
        at = torch.arange(length)
        page, slot = table[at // self.page], at % self.page
        there = (page >= 0) & (page < self.pages)
        page = page.clamp(0, max(self.pages - 1, 0))
        codes = raw(getattr(self.cache, name)).cpu()[page, :, slot].long()
        byte = raw(getattr(self.cache, name + "_scale")).cpu()[page, :, slot].double()
        scale = torch.where(byte == 255, math.nan, torch.exp2(byte - 127))
        return E4M3_OF[codes] * scale[..., None], there


def attention(pr, q, rotate, scale=None, causal=True, window=0, half=2.0 ** -8):
    """(out, error) of every row in 64 bits: `error` is the root mean square that the documented
    roundings leave in the 2-norm of each row (tokens, q_heads).

    A rounding to nearest at relative half step h is off by at most h, h / sqrt(3) in the root mean
    square of a uniform spread, h = 2^-11 for float16.  With w the softmax's weights and O their
    output, a rounding dq of the query moves the output by scale * M dq, M = sum_j w_j (V_j - O) K_j^T,
    and roundings of p by sum_j w_j V_j d_j.  The turn back leaves 2-norms as they are.
    """
    dim, group = pr.dim, q.shape[1] // pr.heads
    scale = dim ** -0.5 if scale is None else scale
    rms = 2.0 ** -11 / math.sqrt(3)
    out = torch.zeros(q.shape, dtype=torch.float64)
    error = torch.zeros(q.shape[:2], dtype=torch.float64)
    starts = pr.starts.cpu().tolist()
    qr = turned(q.cpu(), rotate)
    for b in range(len(starts) - 1):
        (k, there), (v, _) = pr.held("k", b), pr.held("v", b)
        k, v = (torch.where(there[:, None, None], x, 0.0) for x in (k, v))
        length, new = k.shape[0], starts[b + 1] - starts[b]
        if length == 0 or new == 0:
            continue
        bad = ~(torch.isfinite(k) & torch.isfinite(v)).all(-1)  # (length, heads)
        at = length - new + torch.arange(new)[:, None]
        key = torch.arange(length)
        seen = there.expand(new, -1) & (key <= at if causal else True)
        if window:
            seen = seen & (key > at - window)
        rows = slice(starts[b], starts[b + 1])
        for h in range(pr.heads):
            kk, vv = (torch.where(bad[:, h, None], 0.0, x[:, h]) for x in (k, v))
            for g in range(h * group, (h + 1) * group):
                x = qr[rows, g]
                s = (x @ kk.T * scale).masked_fill(~seen, -math.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
                w = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
                o = w @ vv
                wv = w[:, :, None] * (vv[None] - o[:, None])                    # (new, length, dim)
                m = torch.einsum("tjd,je->tde", wv, kk) * scale
                of_q = ((m * x[:, None]) ** 2).sum((1, 2)) * rms ** 2
                of_p = (w ** 2 @ (vv ** 2).sum(-1)) * rms ** 2
                # fp32: scores (dim products, and their size in the exponent), sums of p and p V
                s32 = (x.abs() @ kk.T.abs() * scale).masked_fill(~seen, 0.0).amax(-1)
                of_32 = (2.0 ** -20 * (2 + s32) * (w @ vv.norm(dim=-1))) ** 2
                y = turned(o, rotate)
                error[rows, g] = torch.sqrt(of_q + of_p + of_32 + (half ** 2 / 3) * (y ** 2).sum(-1))
                out[rows, g] = torch.where((seen & bad[:, h]).any(-1, keepdim=True), math.nan, y)
    return out, error


def check_attention(got, pr, q, rotate, dtype, **how):
    """Every row's error in the 2-norm within six times what the roundings leave in the root mean
    square (they are many and independent), zeros and NaN where they belong."""
    want, error = attention(pr, q, rotate, half=HALF_ULP[dtype], **how)
    last = int(pr.starts[-1])
    got, want, error = got.double().cpu()[:last], want[:last], error[:last]
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), (torch.isnan(got) != nan).sum()
    off = torch.where(nan, 0.0, got - want).norm(dim=-1)
    room = 6 * error + TINY[dtype] * pr.dim
    worst = (off / room.clamp(min=1e-300)).max() if off.numel() else 0.0
    assert (off <= room).all(), f"{float(worst) * 6:.2f} times the roundings' root mean square"
    return float(worst) * 6


__all__ = ["Problem", "REALS", "HALF_ULP", "TINY", "attention", "check_attention", "e4m3", "quantised", "raw",
           "turned"]
