"""The feed-forward operators' cases: rotation with 8-bit block quantisation, the product of
8-bit operands with block scales, and the gated projections with their backward pass.

Sizes are generic: widths of 1024 to 8192 (the lengths of 2^10 and 2^12 that the transform's
own configurations have among them), and odd ones between them.  Rows whose length is no
multiple of 16 bytes are views of rows padded to one, as the operators ask for.
"""
import math

import torch

own = False  # set from outside: False computes the plain forms, True calls the framework

BLOCK = 128        # elements that share a scale
E4M3_MAX = 448.0   # the largest finite value of the 8-bit type
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------

def listed():
    return [
        # one token's activations before a down projection in serving: all latency
        {"name": "quantize token", "op": "quantize", "rows": 1, "cols": 8192, "dtype": "bf16",
         "axis": 1, "lines": 1, "rotate": 7},
        # a prompt's activations
        {"name": "quantize prompt", "op": "quantize", "rows": 8192, "cols": 8192,
         "dtype": "bf16", "axis": 1, "lines": 1, "rotate": 7},
        # activations for a weight gradient: blocks down the tokens, an odd number of them
        {"name": "quantize columns", "op": "quantize", "rows": 4099, "cols": 5001,
         "dtype": "f16", "axis": 0, "lines": 1, "rotate": 7},
        # a decode step: one token through a projection, bound by reading the weights
        {"name": "matmul token", "op": "matmul", "m": 1, "n": 4096, "k": 8192, "lines": 128,
         "out": "bf16"},
        # a batch of decoding sequences
        {"name": "matmul batch", "op": "matmul", "m": 48, "n": 8192, "k": 4096, "lines": 128,
         "out": "f16"},
        # a weight gradient with odd sizes: both operands have a scale for each line
        {"name": "matmul ragged", "op": "matmul", "m": 1003, "n": 2057, "k": 1411, "lines": 1,
         "out": "f32"},
        # a prompt or a training batch through a projection
        {"name": "matmul prompt", "op": "matmul", "m": 8192, "n": 8192, "k": 4096, "lines": 128,
         "out": "bf16"},
        # a decode step through both projections
        {"name": "gated token", "op": "gated", "m": 1, "d": 4096, "f": 8192, "dtype": "bf16",
         "act": "silu"},
        # a short prompt, odd sizes
        {"name": "gated ragged", "op": "gated", "m": 333, "d": 1001, "f": 2731, "dtype": "f16",
         "act": "gelu"},
        # a long prompt or a training batch
        {"name": "gated prompt", "op": "gated", "m": 8192, "d": 4096, "f": 8192,
         "dtype": "bf16", "act": "silu"},
        # a training step on a short, odd batch
        {"name": "gated backward ragged", "op": "backward", "m": 517, "d": 1001, "f": 2731,
         "dtype": "f16", "act": "gelu"},
        # a training step
        {"name": "gated backward batch", "op": "backward", "m": 8192, "d": 2048, "f": 8192,
         "dtype": "bf16", "act": "silu"},
    ]


def _size(rng, low, high):
    """A size spread over its logarithm: every third a multiple of 128, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, v // 128 * 128)) if rng.random() < 1 / 3 else v


def draw(rng):
    op = rng.choice(["quantize", "matmul", "gated", "backward"])
    if op == "quantize":
        while True:
            rows, cols = _size(rng, 1, 8192), _size(rng, 128, 8192)
            if rows * cols >= 1024:
                break
        axis, rotate = rng.choice([1, 1, 0]), rng.choice([0, 4, 7])
        return {"op": op, "rows": rows, "cols": cols,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]) if rows * cols <= 1 << 25
                else rng.choice(["bf16", "f16"]),
                "axis": axis, "lines": rng.choice([1, 1, 128]), "rotate": rotate}
    if op == "matmul":
        while True:
            m, n, k = _size(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 8192)
            if m * n * k <= 8192 * 8192 * 4096:
                return {"op": op, "m": m, "n": n, "k": k, "lines": rng.choice([128, 128, 1]),
                        "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
    wide = 4096 if op == "gated" else 2048
    return {"op": op, "m": _size(rng, 1, 8192), "d": _size(rng, 64, wide),
            "f": _size(rng, 64, 8192), "dtype": rng.choice(["bf16", "bf16", "f16"]),
            "act": rng.choice(["silu", "silu", "gelu", "relu"])}


def work(case):
    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        size = DTYPES[case["dtype"]].itemsize
        length, across = (cols, rows) if case["axis"] else (rows, cols)
        scales = -(-length // BLOCK) * -(-across // case["lines"])
        # per element: a butterfly stage a bit, the scaling, the maximum, the product by 1/s
        return {"bytes": rows * cols * (size + 1) + 4 * scales,
                "flops": rows * cols * (case["rotate"] + 3)}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        t = -(-k // BLOCK)
        return {"bytes": m * k + n * k + 4 * t * (m + -(-n // case["lines"]))
                + m * n * DTYPES[case["out"]].itemsize,
                "flops": 2 * m * n * k}
    m, d, f = case["m"], case["d"], case["f"]
    if case["op"] == "gated":
        return {"bytes": 2 * (m * d + 2 * f * d + m * f), "flops": 4 * m * f * d}
    return {"bytes": 2 * (m * f + 2 * m * d + 4 * f * d), "flops": 12 * m * f * d}


# ---- inputs ------------------------------------------------------------------------

def _rows(t, multiple):
    """`t`, its rows padded to a multiple of `multiple` elements where they are not."""
    rows, cols = t.shape
    if cols % multiple == 0:
        return t
    wide = torch.zeros(rows, -(-cols // multiple) * multiple, dtype=t.dtype, device=t.device)
    wide[:, :cols] = t
    return wide[:, :cols]


def _activations(gen, rows, cols, dtype):
    """Normal values with a spread of channel magnitudes and a few outlier channels."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    channel = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    outlier = torch.rand(cols, device="cuda", generator=gen) < 0.004
    return _rows((x * torch.where(outlier, 20.0 * channel, channel)).to(dtype), 16 // dtype.itemsize)


def _weights(gen, rows, cols, dtype):
    w = torch.randn(rows, cols, device="cuda", generator=gen) / math.sqrt(cols)
    return _rows(w.to(dtype), 16 // dtype.itemsize)


def _operand(gen, rows, k, lines):
    """An 8-bit operand with a scale for each block of `lines` x 128."""
    x = torch.randn(rows, k, device="cuda", generator=gen)
    x = x * torch.exp(torch.randn(rows, 1, device="cuda", generator=gen))
    q, scale = _quantize_plain(x, 1, lines, 0)
    return _rows(q.view(torch.uint8), 16).view(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    if case["op"] == "quantize":
        state["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["dtype"]])
    elif case["op"] == "matmul":
        state["a"], state["a_scale"] = _operand(gen, case["m"], case["k"], 1)
        state["b"], state["b_scale"] = _operand(gen, case["n"], case["k"], case["lines"])
    else:
        dtype = DTYPES[case["dtype"]]
        # what follows a norm: unit variance, a moderate spread of the channels
        x = torch.randn(case["m"], case["d"], device="cuda", generator=gen)
        x = x * torch.exp(0.3 * torch.randn(case["d"], device="cuda", generator=gen))
        state["x"] = _rows(x.to(dtype), 8)
        state["w_gate"] = _weights(gen, case["f"], case["d"], dtype)
        state["w_up"] = _weights(gen, case["f"], case["d"], dtype)
        if case["op"] == "backward":
            dh = 0.1 * torch.randn(case["m"], case["f"], device="cuda", generator=gen)
            state["grad"] = _rows(dh.to(dtype), 8)
    return state


# ---- plain forms -------------------------------------------------------------------

def _hadamard(r, dtype):
    """H of size 2^r: (-1)^popc(i & j)."""
    i = torch.arange(1 << r, device="cuda")
    v = i[:, None] & i[None, :]
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = v ^ (v >> 1)
    return (1 - 2 * (v & 1)).to(dtype)


def _blocks(y, lines):
    """y (across, length) zero-extended to whole blocks, as (across / lines, lines, t, 128)."""
    across, length = y.shape
    y = torch.nn.functional.pad(y, (0, -length % BLOCK, 0, -across % lines))
    return y.view(y.shape[0] // lines, lines, y.shape[1] // BLOCK, BLOCK)


def _rotated(y, r):
    """Each aligned group of 2^r along the rows of y by the normalised H, y zero-extended."""
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % (1 << r)))
    if r == 0:
        return y
    return ((y.reshape(-1, 1 << r) @ _hadamard(r, y.dtype)) * 2.0 ** (-r / 2)).view(y.shape)


def _quantize_plain(x, axis, lines, r):
    y = _rotated((x if axis else x.t()).float(), r)
    across, length = y.shape
    y = _blocks(y, lines)
    scale = (y.abs().amax(dim=(1, 3), keepdim=True) / E4M3_MAX).clamp(min=2.0 ** -126)
    q = (y * (1.0 / scale)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(q.shape[0] * lines, -1)[:across, :length]
    return q, scale[:, 0, :, 0]


def _spread(scale, lines, rows, k):
    """A scale for each element of an operand (rows, k)."""
    return scale.repeat_interleave(lines, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :k]


def _activation(g, act):
    """act(g) and act'(g)."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return g * (g > 0), (g > 0).to(g.dtype)


def _plain(s):
    if s["op"] == "quantize":
        return _quantize_plain(s["x"], s["axis"], s["lines"], s["rotate"])
    if s["op"] == "matmul":
        k, lines = s["k"], s["lines"]
        a = s["a"].float() * _spread(s["a_scale"], 1, s["m"], k)
        b = s["b"].float() * _spread(s["b_scale"], lines, s["n"], k)
        return (a @ b.t()).to(DTYPES[s["out"]])
    x, wg, wu, dtype = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["x"].dtype
    g, u = x @ wg.t(), x @ wu.t()
    value, slope = _activation(g, s["act"])
    if s["op"] == "gated":
        return (value * u).to(dtype)
    dh = s["grad"].float()
    dg, du = dh * u * slope, dh * value
    return (dg @ wg + du @ wu).to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)


def _own(s):
    import walsh_hadamard_transform_gb300 as fwt
    if s["op"] == "quantize":
        return fwt.quantize_blocks(s["x"], rotate=s["rotate"], axis=s["axis"], lines=s["lines"])
    if s["op"] == "matmul":
        return fwt.matmul_blocks(s["a"], s["a_scale"], s["b"], s["b_scale"],
                                 out_dtype=DTYPES[s["out"]])
    if s["op"] == "gated":
        return fwt.gated(s["x"], s["w_gate"], s["w_up"], activation=s["act"])
    return fwt.gated_backward(s["grad"], s["x"], s["w_gate"], s["w_up"], activation=s["act"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64 bits -----------------------------------------------------------------------

def _e4m3(v):
    """v (64 bits) rounded to the nearest 8-bit value (3 mantissa bits, least exponent -6), ties to even."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    exponent = torch.where(v.abs() >= 2.0 ** (exponent + 1), exponent + 1, exponent)
    step = 2.0 ** (exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantize(s):
    """Butterflies along the axis, then blocks cut by indexing."""
    y = s["x"].double()
    y = y if s["axis"] else y.t().contiguous()
    r, lines = s["rotate"], s["lines"]
    across, length = y.shape
    full = -(-length // (1 << r)) << r
    y = torch.cat([y, y.new_zeros(across, full - length)], 1)
    for bit in range(r):
        v = y.view(across, -1, 2, 1 << bit)
        y = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).view(across, full)
    y = y / math.sqrt(2.0 ** r)
    row = torch.arange(across, device=y.device) // lines
    col = torch.arange(full, device=y.device) // BLOCK
    top = y.new_zeros(int(row[-1]) + 1, full).index_reduce(0, row, y.abs(), "amax")
    top = top.new_zeros(top.shape[0], int(col[-1]) + 1).index_reduce(1, col, top, "amax")
    scale = torch.clamp(top / E4M3_MAX, min=2.0 ** -126)
    return _e4m3(y / scale[row][:, col]), scale


def _exact_matmul(s):
    m, n, k = s["m"], s["n"], s["k"]
    c = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for t, k0 in enumerate(range(0, k, BLOCK)):
        a, b = s["a"][:, k0:k0 + BLOCK].double(), s["b"][:, k0:k0 + BLOCK].double()
        row = torch.arange(n, device="cuda") // s["lines"]
        c += (a * s["a_scale"][:, t:t + 1].double()) @ (b * s["b_scale"][row, t:t + 1].double()).T
    return c


def _exact_gated(s):
    x, wg, wu = (s[name].double() for name in ("x", "w_gate", "w_up"))
    g, u = torch.einsum("md,fd->mf", x, wg), torch.einsum("md,fd->mf", x, wu)
    if s["act"] == "silu":
        p = torch.sigmoid(g)
        value, slope = g * p, p + g * p * (1 - p)
    elif s["act"] == "gelu":
        # tanh(z) = 2 sigmoid(2 z) - 1, so the half-sum is sigmoid(2 z)
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (g + 0.044715 * g ** 3))
        value, slope = g * p, p + g * p * (1 - p) * c * (1 + 0.134145 * g ** 2)
    else:
        value, slope = g.clamp(min=0), torch.heaviside(g, torch.zeros_like(g))
    if s["op"] == "gated":
        return value * u
    dh = s["grad"].double()
    dg, du = dh * u * slope, dh * value
    return (torch.einsum("mf,fd->md", dg, wg) + torch.einsum("mf,fd->md", du, wu),
            torch.einsum("mf,md->fd", dg, x), torch.einsum("mf,md->fd", du, x))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(s)
    if case["op"] == "matmul":
        return _exact_matmul(s)
    return _exact_gated(s)
