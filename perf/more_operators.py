"""The cache operators' cases: keys and values rotated and held in 8 bits in pages, written as
tokens come (`cache_append`), read back (`cache_read`), and attended to by the newest tokens of
each sequence (`cache_attention`), from single tokens to whole prompts.

A cache is four tensors: codes e4m3 (pages, heads, tokens of a page, dim) of keys and of values,
and for each a scale (pages, heads, tokens of a page), a power of two held in e8m0.  `table`
(sequences, most pages) names each sequence's pages in order; `lengths` are the tokens that each
sequence has in the cache, and rows starts[b] to starts[b + 1] of the packed inputs and outputs
are the last of them.  Sizes are generic: heads of 64 and 128, pages of 16 to 128 tokens.
"""
import math
import random

import torch

own = False  # set from outside: False computes the plain forms, True calls the framework

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------

def _case(op, sequences, new, context, heads, dim, page, dtype, group=1, spread=0, singles=0,
          rotate=-1, causal=True, window=0):
    """`sequences` of up to `new` new tokens and `context` in all, and `singles` more with one new
    token; spread: 0 for all alike, else a number that draws their sizes.  rotate: -1, whole heads."""
    return {"op": op, "sequences": sequences, "new": new, "context": context, "heads": heads,
            "group": group, "dim": dim, "page": page, "dtype": dtype, "spread": spread,
            "singles": singles, "rotate": rotate, "causal": causal, "window": window}


def listed():
    return [
        # a decode step of 64 sequences: each writes one token; all latency
        {"name": "append tokens", **_case("append", 64, 1, 4096, 8, 128, 16, "bf16", spread=1)},
        # a prompt's keys and values
        {"name": "append prompt", **_case("append", 1, 8192, 8192, 8, 128, 64, "bf16")},
        # chunks of several prompts, small heads in an odd number
        {"name": "append ragged", **_case("append", 9, 700, 5000, 5, 64, 32, "f16", spread=2,
                                          rotate=4)},
        # a shared prefix read back for another program
        {"name": "read prefix", **_case("read", 4, 4096, 4096, 8, 128, 64, "bf16")},
        # the last tokens of some sequences, in 32 bits
        {"name": "read ragged", **_case("read", 7, 1500, 5000, 3, 64, 16, "f32", spread=3)},
        # one user's decode step: latency
        {"name": "attention token", **_case("attention", 1, 1, 4099, 8, 128, 16, "bf16", group=4)},
        # a batch of decoding sequences of all lengths: bound by reading the cache
        {"name": "attention batch", **_case("attention", 64, 1, 16384, 8, 128, 64, "bf16", group=4,
                                            spread=4)},
        # drafted tokens checked at once, under a sliding window
        {"name": "attention drafts", **_case("attention", 16, 5, 6000, 4, 64, 16, "f16", group=2,
                                             spread=5, window=1024)},
        # odd chunks of several prompts beside their contexts
        {"name": "attention ragged", **_case("attention", 5, 701, 5003, 5, 64, 32, "f16", group=3,
                                             spread=6, rotate=4)},
        # a step of a server: one prompt's chunk among decoding sequences
        {"name": "attention mix", **_case("attention", 1, 512, 4096, 8, 128, 64, "bf16", group=4,
                                          singles=32, spread=7)},
        # a whole prompt, a key head to each query head
        {"name": "attention prompt", **_case("attention", 1, 8192, 8192, 16, 128, 64, "bf16")},
        # a chunk of a long prompt
        {"name": "attention chunk", **_case("attention", 1, 4096, 32768, 8, 128, 128, "bf16",
                                            group=4)},
    ]


def _size(rng, low, high):
    """A size spread over its logarithm: every third a multiple of 64, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = max(low, v // 64 * 64) if rng.random() < 1 / 3 else v
    return min(high, v)


def draw(rng):
    most = work(listed()[-1])
    while True:
        op = rng.choice(["append", "read", "token", "chunk", "chunk"])
        context = _size(rng, 16, 32768)
        sequences = rng.choice([1, 1, 2, 3, 5, 16, 33, 64])
        new = rng.choice([1, 1, 1, 2, 5]) if op == "token" else _size(rng, 1, 8192)
        new = min(new, context)
        dim = rng.choice([64, 128, 128])
        case = _case("attention" if op in ("token", "chunk") else op, sequences, new, context,
                     heads=rng.choice([1, 2, 3, 5, 8, 8, 16]), dim=dim,
                     page=rng.choice([16, 32, 64, 128]),
                     dtype=rng.choice(["bf16", "bf16", "f16"] if op in ("token", "chunk")
                                      else ["bf16", "bf16", "f16", "f32"]),
                     group=rng.choice([1, 2, 3, 4, 4, 8]) if op in ("token", "chunk") else 1,
                     spread=rng.choice([0, rng.randrange(1, 1 << 20)]),
                     singles=rng.choice([0, 0, 0, rng.randrange(1, 40)]),
                     rotate=rng.choice([-1, -1, 0, 4]),
                     causal=rng.random() < 0.85,
                     window=rng.choice([0, 0, 0, _size(rng, 1, 8192)]))
        if op in ("append", "read"):
            case["causal"], case["window"] = True, 0
        news, lens = _lengths(case)
        w = work(case)
        # (the plain form spreads ragged sequences out to the longest, in both directions)
        scores = len(news) * case["heads"] * case["group"] * max(news) * max(lens)
        cache = len(news) * max(lens) * case["heads"] * dim
        tokens = sum(news) * case["heads"] * dim
        if (1e4 < w["bytes"] <= 1.2e9 and w["flops"] <= most["flops"] and scores <= 4.3e9
                and cache <= 1.1e9 and sum(lens) <= 1 << 20
                and (case["op"] == "attention" or 4096 <= tokens <= 1 << 25)):
            return case


def _lengths(case):
    """New tokens and all tokens of each sequence."""
    rng = random.Random(case["spread"])
    news, lens = [], []
    for i in range(case["sequences"]):
        new, length = case["new"], case["context"]
        if case["spread"] and i:
            new = int(math.exp(rng.uniform(0, math.log(new)))) if new > 1 else 1
            length = int(math.exp(rng.uniform(math.log(max(new, length // 64)), math.log(length))))
            length = min(case["context"], max(new, length))
        news.append(new)
        lens.append(length)
    for i in range(case["singles"]):
        news.append(1)
        lens.append(rng.randrange(max(1, case["context"] // 4), case["context"] + 1))
    return news, lens


def _seen(new, length, case):
    """(keys that some new token sees, pairs of a new token and a key that it sees)."""
    pairs, first = 0, length
    for t in range(new):
        high = length - new + t + 1 if case["causal"] else length
        low = max(0, length - new + t + 1 - case["window"]) if case["window"] else 0
        pairs += max(0, high - low)
        first = min(first, low)
    return length - first, pairs


def work(case):
    news, lens = _lengths(case)
    heads, dim, tokens = case["heads"], case["dim"], sum(news)
    size = DTYPES[case["dtype"]].itemsize
    index = 4 * (2 * len(news) + 1 + sum(-(-n // case["page"]) for n in lens))
    if case["op"] != "attention":
        rotate = int(math.log2(dim)) if case["rotate"] < 0 else case["rotate"]
        each = 2 * heads * dim * tokens
        return {"bytes": each * (size + 1) + 2 * heads * tokens + index,
                "flops": each * (rotate + 3)}
    keys = pairs = 0
    for new, length in zip(news, lens):
        k, p = _seen(new, length, case)
        keys, pairs = keys + k, pairs + p
    return {"bytes": 2 * tokens * heads * case["group"] * dim * size
            + keys * heads * (2 * dim + 2) + index,
            "flops": 4 * dim * heads * case["group"] * pairs}


# ---- inputs ------------------------------------------------------------------------

def _vectors(gen, tokens, heads, dim, outliers):
    """Normal values with a spread of channel magnitudes; keys have a few outlier channels."""
    x = torch.randn(tokens, heads, dim, device="cuda", generator=gen)
    channel = torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=gen))
    if outliers:
        channel = torch.where(torch.rand(heads, dim, device="cuda", generator=gen) < 0.02,
                              8 * channel, channel)
    return x * channel


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    news, lens = _lengths(case)
    heads, dim, page, dtype = case["heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    rotate = int(math.log2(dim)) if case["rotate"] < 0 else case["rotate"]
    tokens, counts = sum(news), [-(-n // page) for n in lens]
    # pages in any order, as a server's free list hands them out; some belong to nobody
    pages = sum(counts) + 3
    order = torch.randperm(pages, device="cuda", generator=gen)[:sum(counts)].to(torch.int32)
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    ends = [0]
    for n in news:
        ends.append(ends[-1] + n)
    state.update(rotate=rotate, tokens=tokens, table=table, most_new=max(news), most=max(lens),
                 starts=torch.tensor(ends, dtype=torch.int32, device="cuda"),
                 lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    append = case["op"] == "append"
    # slots that hold nothing yet are zero, or, where the cache is read, whatever was there
    cache = {name: torch.full((pages, heads, page) + ((dim,) if name in "kv" else ()),
                              0 if append else 0x7f if name in "kv" else 0xff,
                              dtype=torch.uint8, device="cuda")
             for name in ("k", "k_scale", "v", "v_scale")}
    if append:
        state["k"] = _vectors(gen, tokens, heads, dim, True).to(dtype)
        state["v"] = _vectors(gen, tokens, heads, dim, False).to(dtype)
    else:
        for b, n in enumerate(lens):
            slots = torch.arange(n, device="cuda")
            where, slot = table[b][slots // page].long(), slots % page
            for name in ("k", "v"):
                x = _vectors(gen, n, heads, dim, name == "k").bfloat16()
                codes, scale = _quantised(x, rotate)
                cache[name][where, :, slot] = codes
                cache[name + "_scale"][where, :, slot] = scale
    if case["op"] == "attention":
        q = _vectors(gen, tokens, heads * case["group"], dim, False)
        state["q"] = (0.7 * q).to(dtype)
    state["cache"] = {name: t.view(torch.float8_e4m3fn if name in "kv" else torch.float8_e8m0fnu)
                      for name, t in cache.items()}
    return state


# ---- plain forms -------------------------------------------------------------------

def _rotated(x, r):
    """Each aligned group of 2^r along the last dimension by the normalised H."""
    if r == 0:
        return x
    i = torch.arange(1 << r, device=x.device)
    v = i[:, None] & i[None, :]
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = v ^ (v >> 1)
    h = (1 - 2 * (v & 1)).to(x.dtype) * 2.0 ** (-r / 2)
    return (x.reshape(-1, 1 << r) @ h).view(x.shape)


def _quantised(x, r):
    """Codes of the rotated x (tokens, heads, dim) and its scales 2^(s - 127), s the least from 1 on
    for which the largest magnitude is at most 448 times the scale, both as bytes."""
    y = _rotated(x.float(), r)
    top = y.abs().amax(-1)
    m, e = torch.frexp(top.clamp(min=2.0 ** -118))      # 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    y = torch.ldexp(y, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _places(s):
    """Sequence, position, page and slot of each row of the packed tensors."""
    row = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["starts"][1:], row, right=True)
    at = (s["lengths"][b] - s["starts"][b + 1] + row).long()
    return b, at, s["table"][b, at // s["page"]].long(), at % s["page"]


def _values(s, name, page, slot):
    """What the cache holds there, in 32 bits, still rotated: (..., heads, dim)."""
    codes = s["cache"][name].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    power = s["cache"][name + "_scale"].view(torch.uint8)[page, :, slot].int() - 127
    return torch.ldexp(codes, power[..., None])


def _append_plain(s):
    _, _, page, slot = _places(s)
    for name in ("k", "v"):
        codes, scale = _quantised(s[name], s["rotate"])
        s["cache"][name].view(torch.uint8)[page, :, slot] = codes
        s["cache"][name + "_scale"].view(torch.uint8)[page, :, slot] = scale
    return s["cache"]


def _read_plain(s):
    _, _, page, slot = _places(s)
    return tuple(_rotated(_values(s, name, page, slot), s["rotate"]).to(DTYPES[s["dtype"]])
                 for name in ("k", "v"))


def _attention_plain(s):
    heads, group, dim, dtype = s["heads"], s["group"], s["dim"], DTYPES[s["dtype"]]
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    length, batch = s["lengths"].long(), s["lengths"].numel()
    key = torch.arange(s["most"], device="cuda")
    page = s["table"][:, key // s["page"]].long().clamp(min=0)
    there = (key < length[:, None])[..., None, None]
    slot = (key % s["page"]).expand_as(page)
    k, v = (torch.where(there, _values(s, name, page, slot), 0.0).permute(0, 2, 1, 3)
            for name in ("k", "v"))                                  # (batch, heads, most, dim)
    t = torch.arange(s["most_new"], device="cuda")
    row = (s["starts"][:-1, None] + t).clamp(max=s["tokens"] - 1).long()
    q = _rotated(s["q"].float(), s["rotate"])[row].view(batch, -1, heads, group, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)      # (batch, heads, group * t, dim)
    score = (q @ k.transpose(2, 3) * dim ** -0.5).view(batch, heads, group, -1, s["most"])
    last = (length - new)[:, None] + t                               # the token's own position
    seen = (key < length[:, None])[:, None].expand(-1, len(t), -1)
    if s["causal"]:
        seen = seen & (key <= last[..., None])
    if s["window"]:
        seen = seen & (key > last[..., None] - s["window"])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    del score
    total = p.sum(-1, keepdim=True)
    out = (p.view(batch, heads, -1, s["most"]) @ v).view(*p.shape[:-1], dim)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, len(t), heads * group, dim)
    b, at, _, _ = _places(s)
    return _rotated(out[b, at - (length - new)[b]], s["rotate"]).to(dtype)


def _plain(s):
    if s["op"] == "append":
        return _append_plain(s)
    return _read_plain(s) if s["op"] == "read" else _attention_plain(s)


def _own(s):
    import walsh_hadamard_transform_gb300 as fwt
    cache = fwt.Cache(**s["cache"])
    place = (cache, s["table"], s["starts"], s["lengths"])
    if s["op"] == "append":
        fwt.cache_append(s["k"], s["v"], *place, rotate=s["rotate"])
        return s["cache"]
    if s["op"] == "read":
        return fwt.cache_read(*place, s["tokens"], dtype=DTYPES[s["dtype"]], rotate=s["rotate"])
    return fwt.cache_attention(s["q"], *place, rotate=s["rotate"], causal=s["causal"],
                               window=s["window"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64 bits -----------------------------------------------------------------------

def _turned(y, r):
    """The rotation by butterflies, in 64 bits."""
    shape = y.shape
    y = y.double().reshape(-1, shape[-1])
    for bit in range(r):
        v = y.view(y.shape[0], -1, 2, 1 << bit)
        y = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).view(y.shape[0], -1)
    return (y / math.sqrt(2.0 ** r)).view(shape)


def _held(s, name, b, first, count):
    """Tokens first .. first + count - 1 of sequence b as the cache holds them, in 64 bits."""
    at = torch.arange(first, first + count, device="cuda")
    page, slot = s["table"][b].long()[at // s["page"]], at % s["page"]
    code = torch.arange(256, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    raw = s["cache"][name].view(torch.uint8)[page, :, slot].long()
    power = s["cache"][name + "_scale"].view(torch.uint8)[page, :, slot].double() - 127
    return code[raw] * torch.exp2(power)[..., None]


def _exact_append(s):
    out = {name: t.double() for name, t in s["cache"].items()}
    starts, lens = s["starts"].tolist(), s["lengths"].tolist()
    for b, length in enumerate(lens):
        count = starts[b + 1] - starts[b]
        at = torch.arange(length - count, length, device="cuda")
        page, slot = s["table"][b].long()[at // s["page"]], at % s["page"]
        for name in ("k", "v"):
            y = _turned(s[name][starts[b]:starts[b + 1]], s["rotate"])
            scale = y.abs().amax(-1, keepdim=True) / E4M3_MAX
            power = torch.ceil(torch.log2(scale.clamp(min=2.0 ** -126)))
            y = y / torch.exp2(power)
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            out[name][page, :, slot] = torch.round(y / step) * step
            out[name + "_scale"][page, :, slot] = torch.exp2(power[..., 0])
    return out


def _exact_read(s):
    starts, lens = s["starts"].tolist(), s["lengths"].tolist()
    rows = {"k": [], "v": []}
    for b, length in enumerate(lens):
        count = starts[b + 1] - starts[b]
        for name in rows:
            rows[name].append(_turned(_held(s, name, b, length - count, count), s["rotate"]))
    return torch.cat(rows["k"]), torch.cat(rows["v"])


def _exact_attention(s):
    """Keys and values turned back, and each query head by itself, a stretch of tokens at a time."""
    starts, lens, group, dim = s["starts"].tolist(), s["lengths"].tolist(), s["group"], s["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        k, v = (_turned(_held(s, name, b, 0, length), s["rotate"]) for name in ("k", "v"))
        new = starts[b + 1] - starts[b]
        key = torch.arange(length, device="cuda")
        for h in range(s["heads"]):
            for first in range(0, new, 4096):
                t = torch.arange(first, min(first + 4096, new), device="cuda")
                q = s["q"][starts[b] + first:starts[b] + first + len(t),
                           h * group:(h + 1) * group].double()
                own_at = (length - new + t)[:, None]
                hidden = torch.zeros(len(t), length, dtype=torch.bool, device="cuda")
                if s["causal"]:
                    hidden |= key > own_at
                if s["window"]:
                    hidden |= key <= own_at - s["window"]
                z = torch.einsum("tgd,kd->tgk", q, k[:, h]) / math.sqrt(dim)
                z = z.masked_fill(hidden[:, None], -math.inf)
                z = torch.exp(z - z.amax(-1, keepdim=True))
                o = torch.einsum("tgk,kd->tgd", z, v[:, h]) / z.sum(-1, keepdim=True)
                out[starts[b] + first:starts[b] + first + len(t), h * group:(h + 1) * group] = o
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_read(s) if case["op"] == "read" else _exact_attention(s)
