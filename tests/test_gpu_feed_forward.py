"""The feed-forward operators on the GPU against their definitions in 64 bits.

Tolerances follow from the arithmetic.  With u = 2^-24 (fp32's half unit in the last
place), a sum of k products held in 32 bits, rounded or truncated at each step, is
within k * 2u of the exact one relative to the sum of the products' magnitudes; an
output rounded to fewer bits adds its own half unit in the last place.
"""
import math

import pytest
import torch

import feed_forward_plain as plain
import walsh_hadamard_transform_gb300 as fwt
from feed_forward_plain import HALF_ULP, REALS, TINY

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def window(values, dtype, multiple, extra=0):
    """values as a CUDA window of a matrix whose other elements are NaN; rows a multiple of
    `multiple` elements apart."""
    rows, cols = values.shape
    ld = cols + (-cols % multiple) + extra * multiple
    wide = torch.full((rows + 2, ld), NAN, dtype=torch.float32).to(dtype).cuda()
    out = wide[1:rows + 1, :cols]
    if dtype == torch.float8_e4m3fn:
        out.view(torch.uint8).copy_(values.to(dtype).view(torch.uint8))
    else:
        out.copy_(values.to(dtype))
    return out, wide


def untouched(out, wide):
    """Whether nothing but `out` was written in `wide`."""
    rows, cols = out.shape
    rest = wide.float().clone()
    rest[1:rows + 1, :cols] = NAN
    return bool(torch.isnan(rest).all())


def activations(rows, cols, seed, outliers=True):
    x = torch.randn(rows, cols, generator=gen(seed), dtype=torch.float64)
    if outliers and cols > 3:
        x[:, 2] *= 30
    return x


# ---- quantize_blocks ---------------------------------------------------------------

QUANTIZE = [  # rows, cols, dtype, rotate, axis, lines
    (1, 128, "bf16", 7, 1, 1), (1, 8192, "bf16", 7, 1, 1), (3, 1, "bf16", 0, 1, 1),
    (17, 129, "bf16", 0, 1, 1), (33, 1000, "f16", 3, 1, 1), (16, 640, "f32", 7, 1, 1),
    (5, 131, "f32", 1, 1, 1), (130, 257, "bf16", 5, 1, 128), (128, 384, "f16", 7, 1, 128),
    (300, 72, "bf16", 7, 0, 1), (1, 40, "f16", 2, 0, 1), (129, 200, "f32", 6, 0, 1),
    (257, 130, "bf16", 4, 0, 128), (515, 1024, "f16", 7, 0, 1), (64, 100, "f32", 7, 0, 128),
    (100, 4096, "bf16", 2, 1, 1), (2, 300, "bf16", 7, 0, 1),
]


def check_quantized(x, q, scale, r, axis, lines):
    y = plain.rotated(x, r, axis)
    rows, length = y.shape
    assert q.shape == (rows, length)
    # the rotation: r stages of fp32 sums of the group's magnitudes
    slack = (r + 2) * 2 * U * plain.rotated(x.double().cpu().abs(), 0, axis)
    slack = torch.nn.functional.pad(slack, (0, length - slack.shape[1]))
    group = 1 << r
    slack = slack.view(rows, -1, group).sum(2, keepdim=True).expand(-1, -1, group)
    slack = slack.reshape(rows, length) * 2.0 ** (-r / 2)
    top = plain.block_max(y, lines)
    got = scale.double().cpu()
    want = (top / 448).clamp(min=2.0 ** -126)
    loose = plain.block_max(slack, lines) / 448 + 2 * U * want
    assert ((got - want).abs() <= loose).all()
    s = plain.spread(scale, lines, rows, length)
    v = plain.values(q)
    # a code lies between those of the ends of y * (1 / s)'s fp32 error: exact but next to a tie
    reach = slack + 8 * U * y.abs()
    assert (v >= plain.e4m3((y - reach) / s)).all() and (v <= plain.e4m3((y + reach) / s)).all()


@pytest.mark.parametrize("rows,cols,dtype,rotate,axis,lines", QUANTIZE)
@pytest.mark.parametrize("aligned", [True, False])
def test_quantize_blocks(rows, cols, dtype, rotate, axis, lines, aligned):
    dt = REALS[dtype]
    if aligned:
        x, _ = window(activations(rows, cols, rows + cols), dt, 16 // dt.itemsize)
    else:  # rows of elements' alignment only
        x = window(activations(rows, cols, rows + cols), dt, 1, extra=cols % 2 * 2 + 1)[0]
    across, length = (rows, cols) if axis else (cols, rows)
    length += -length % (1 << rotate)
    q, qw = window(torch.zeros(across, length), torch.float8_e4m3fn, 16, extra=1)
    s, sw = window(torch.zeros(-(-across // lines), -(-length // 128)), torch.float32, 1, extra=3)
    got = fwt.quantize_blocks(x, rotate=rotate, axis=axis, lines=lines, out=(q, s))
    assert got[0] is q and got[1] is s
    check_quantized(x, q, s, rotate, axis, lines)
    assert untouched(q, qw) and untouched(s, sw)
    q2, s2 = fwt.quantize_blocks(x, rotate=rotate, axis=axis, lines=lines)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


def test_quantize_special_values():
    x = torch.zeros(20, 512)
    x[0, 0] = 1.0            # alone in its block
    x[1, 130] = float("inf")
    x[2, 300] = NAN
    x[3, 5] = 2.0 ** -140    # below the smallest scale's smallest code
    x[4, :] = 3.0e38         # overflows in the rotation
    x[5, 7] = -448.0
    q, s = fwt.quantize_blocks(x.cuda(), rotate=7)
    v, s = plain.values(q), s.cpu()
    assert (s[6:] == 2.0 ** -126).all() and (v[6:] == 0).all()
    assert torch.isnan(s).nonzero().tolist() == [[1, 1], [2, 2], [4, 0], [4, 1], [4, 2], [4, 3]]
    bad = torch.isnan(s).repeat_interleave(128, 1)
    assert torch.isnan(v[bad]).all() and not torch.isnan(v[~bad]).any()
    assert (v[0, :128] == 448).all() and (v[0, 128:] == 0).all()
    assert (v[3] == 0).all()
    q, s = fwt.quantize_blocks(x.cuda(), rotate=0)
    v, s = plain.values(q), s.cpu()
    assert torch.isnan(s).nonzero().tolist() == [[1, 1], [2, 2]]
    assert v[5, 7] == -448 and v[5].abs().sum() == 448 and s[5, 0] == 1.0


def test_quantize_ties_go_to_even():
    v = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 0.0009765625, 0.0029296875, 17.0, 19.0] * 16)
    q, s = fwt.quantize_blocks(v.view(1, 128).cuda(), rotate=0)
    assert s.item() == 1.0
    assert plain.values(q)[0, :8].tolist() == [448, 1.0, 1.25, -1.0, 0, 0.00390625, 16, 20]


def test_quantize_offsets_beyond_32_bits():
    ld = (1 << 30) + 8  # rows two and three start past 2^31 bytes and 2^31 elements
    wide = torch.empty(2 * ld + 256, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((3, 256), (ld, 1))
    x.copy_(activations(3, 256, 5))
    q, s = fwt.quantize_blocks(x, rotate=7)
    check_quantized(x, q, s, 7, 1, 1)


@pytest.mark.parametrize("axis,lines", [(1, 1), (1, 128), (0, 1), (0, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_large_calls_equal_their_parts(axis, lines, dtype):
    """Large calls go through several blocks a warp, small ones through one: the same bits."""
    rows, cols = (4099, 10250) if axis else (10250, 4099)
    x = torch.randn(rows, cols + -cols % 8, device="cuda").to(REALS[dtype])[:, :cols]
    q, s = fwt.quantize_blocks(x, rotate=5, axis=axis, lines=lines)
    across = q.shape[0]
    for start, size in ((0, 256), (1792, 128), (4096, across - 4096)):
        part = x[start:start + size] if axis else x[:, start:start + size]
        qp, sp = fwt.quantize_blocks(part, rotate=5, axis=axis, lines=lines)
        assert torch.equal(qp.view(torch.uint8), q[start:start + size].view(torch.uint8))
        assert torch.equal(sp, s[start // lines:start // lines + sp.shape[0]])


# ---- matmul_blocks -----------------------------------------------------------------

def operand(rows, k, lines, seed, extra=0):
    x = torch.randn(rows, k, generator=gen(seed)) * torch.exp(torch.randn(rows, 1, generator=gen(seed + 1)))
    top = plain.block_max(x.double(), lines)
    scale = (top / 448).float().clamp(min=2.0 ** -126)
    q = plain.e4m3(x.double() / plain.spread(scale, lines, rows, k))
    return (window(q.float(), torch.float8_e4m3fn, 16, extra)[0],
            window(scale, torch.float32, 1, extra)[0])


def matmul_expected(a, sa, b, sb, lines):
    k = a.shape[1]
    x = plain.values(a) * plain.spread(sa, 1, a.shape[0], k)
    y = plain.values(b) * plain.spread(sb, lines, b.shape[0], k)
    return x @ y.t(), x.abs() @ y.abs().t()


MATMUL = [  # m, n, k, lines, out
    (1, 1, 1, 1, "f32"), (1, 128, 128, 128, "f32"), (1, 4096, 1024, 128, "bf16"),
    (2, 100, 1000, 128, "f16"), (7, 333, 515, 128, "f32"), (8, 512, 2048, 1, "f32"),
    (16, 1024, 4096, 128, "bf16"), (17, 257, 129, 1, "f32"), (33, 640, 272, 128, "f16"),
    (64, 2000, 1500, 128, "f32"), (100, 130, 4000, 1, "bf16"), (128, 128, 64, 128, "f32"),
    (129, 300, 700, 128, "f32"), (200, 1100, 1152, 1, "f32"), (257, 2057, 385, 1, "f16"),
    (300, 513, 2049, 128, "bf16"), (1024, 1024, 1024, 128, "f32"), (1500, 3000, 640, 128, "bf16"),
    (3, 50000, 160, 128, "bf16"), (4000, 5, 200, 1, "f32"), (640, 384, 1, 128, "f32"),
    (2307, 2500, 400, 128, "bf16"), (2500, 2307, 261, 1, "f32"), (2049, 2560, 640, 128, "f16"),
    (150, 2500, 900, 128, "bf16"), (129, 1290, 1700, 1, "f32"), (50, 2600, 1600, 128, "f16"),
    (200, 3800, 2500, 1, "bf16"), (300, 1700, 2600, 128, "f32"), (130, 1900, 2000, 128, "f16"),
    (40, 7000, 2600, 128, "bf16"), (300, 9800, 200, 128, "bf16"), (300, 9800, 200, 1, "f16"),
]


@pytest.mark.parametrize("m,n,k,lines,out", MATMUL)
def test_matmul_blocks(m, n, k, lines, out):
    a, sa = operand(m, k, 1, m + k, extra=1)
    b, sb = operand(n, k, lines, n + 7 * k, extra=2)
    c, cw = window(torch.zeros(m, n), REALS[out], 16 // REALS[out].itemsize, extra=1)
    assert fwt.matmul_blocks(a, sa, b, sb, out=c) is c
    want, size = matmul_expected(a, sa, b, sb, lines)
    bound = (min(k, 128) + -(-k // 128) + 3) * 2 * U * size + HALF_ULP[out] * want.abs() + TINY[out]
    err = (c.double().cpu() - want).abs()
    assert (err <= bound).all(), (err / bound.clamp(min=1e-300)).max()
    assert untouched(c, cw)
    # an output whose rows start anywhere, and the same bits again
    odd, oddw = window(torch.zeros(m, n), REALS[out], 1, extra=n % 2 + 2)
    fwt.matmul_blocks(a, sa, b, sb, out=odd)
    assert torch.equal(odd, c) and untouched(odd, oddw)
    made = fwt.matmul_blocks(a, sa, b, sb, out_dtype=REALS[out])
    assert torch.equal(made, c)


@pytest.mark.parametrize("m,n,k", [(5, 300, 400), (40, 200, 300), (300, 400, 500)])
@pytest.mark.parametrize("lines", [1, 128])
def test_matmul_special_values_stay_in_their_rows_and_columns(m, n, k, lines):
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, lines, 2)
    clean = fwt.matmul_blocks(a, sa, b, sb, out_dtype=torch.float32)
    a.view(torch.uint8)[3, 200] = 0x7f  # NaN
    sa[1, 1] = NAN
    b.view(torch.uint8)[150, 7] = 0xff
    out = fwt.matmul_blocks(a, sa, b, sb, out_dtype=torch.float32)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[1] = bad[3] = True
    bad[:, 150] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[~bad])


def test_matmul_over_nothing():
    a, sa = torch.empty(5, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, 0, device="cuda")
    b, sb = torch.empty(9, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(9, 0, device="cuda")
    c, cw = window(torch.ones(5, 9), torch.float32, 4)
    fwt.matmul_blocks(a, sa, b, sb, out=c)
    assert (c == 0).all() and untouched(c, cw)
    a, sa = operand(3, 128, 1, 1)
    e, se = torch.empty(0, 128, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(0, 1, device="cuda")
    assert fwt.matmul_blocks(a, sa, e, se).shape == (3, 0)
    assert fwt.matmul_blocks(e, se, a, sa).shape == (0, 3)


def test_rotation_of_both_operands_leaves_the_product():
    x, w = activations(200, 768, 1), activations(300, 768, 2, outliers=False)
    exact = x @ w.t()
    errors = []
    for r in (0, 7):
        a = fwt.quantize_blocks(x.float().cuda(), rotate=r)
        b = fwt.quantize_blocks(w.float().cuda(), rotate=r, lines=128)
        c = fwt.matmul_blocks(*a, *b, out_dtype=torch.float32).double().cpu()
        errors.append(((c - exact).norm() / exact.norm()).item())
    # e4m3 keeps 4 significant bits: a relative error of at most 2^-4 an operand, uniform
    # within a step, so 2^-4 / sqrt(3) each at the worst
    assert max(errors) <= 2 * 2.0 ** -4 / math.sqrt(3)


# ---- gated -------------------------------------------------------------------------

GATED = [  # m, d, f, dtype, act
    (1, 8, 1, "bf16", "silu"), (1, 1024, 4096, "bf16", "silu"), (1, 1001, 333, "f16", "gelu"),
    (2, 64, 130, "f16", "relu"), (5, 520, 1000, "bf16", "gelu"), (8, 2048, 512, "bf16", "silu"),
    (9, 100, 257, "f16", "silu"), (16, 1024, 640, "bf16", "relu"), (17, 72, 2000, "f16", "gelu"),
    (40, 640, 384, "bf16", "silu"), (64, 1000, 1000, "f16", "silu"), (128, 64, 128, "bf16", "gelu"),
    (129, 1001, 531, "f16", "gelu"), (333, 200, 1031, "bf16", "silu"), (700, 513, 900, "bf16", "relu"),
    (1030, 1024, 1024, "f16", "silu"), (3, 1, 5, "bf16", "silu"), (130, 3, 70, "f16", "silu"),
    (100, 1500, 2000, "bf16", "gelu"), (200, 1800, 1500, "f16", "silu"), (129, 1600, 1200, "bf16", "silu"),
    (300, 72, 4900, "bf16", "silu"),
    (1500, 200, 2105, "bf16", "gelu"), (1281, 513, 3000, "f16", "silu"),
]


def gated_inputs(m, d, f, dtype, extra=0):
    dt = REALS[dtype]
    make = lambda rows, cols, seed, scale: window(  # noqa: E731
        torch.randn(rows, cols, generator=gen(seed), dtype=torch.float64) * scale, dt, 8, extra)[0]
    return (make(m, d, m + d, 1.0), make(f, d, f, 2 / math.sqrt(d)), make(f, d, f + 1, 1 / math.sqrt(d)),
            make(m, f, m + f, 0.1))


def gated_slack(x, wg, wu, act):
    """Bounds of the fp32 errors of the products g and u, of act(g) and of act'(g)."""
    x, wg, wu = (t.double().cpu() for t in (x, wg, wu))
    k = x.shape[1]
    g = x @ wg.t()
    eg, eu = k * 2 * U * (x.abs() @ wg.abs().t()), k * 2 * U * (x.abs() @ wu.abs().t())
    # |act'| <= 1.13, |act''| <= 1.2 for all three but relu's step; the exponential is good
    # to 2^-21 relative and |g| 2^-23 for its argument's rounding, and the logistic so too
    rough = (2.0 ** -20 + (g.abs() + 0.045 * g.abs() ** 3).clamp(max=100) * 2.0 ** -22)
    value = 1.13 * eg + g.abs() * rough + 1e-37
    slope = 1.2 * eg + (1 + 2 * g.abs()) * rough + 1e-37
    if act == "relu":
        slope = (g.abs() <= eg).double()
    return eg, eu, value, slope


@pytest.mark.parametrize("m,d,f,dtype,act", GATED)
def test_gated(m, d, f, dtype, act):
    x, wg, wu, _ = gated_inputs(m, d, f, dtype, extra=1)
    h, hw = window(torch.zeros(m, f), REALS[dtype], 8, extra=1)
    assert fwt.gated(x, wg, wu, activation=act, out=h) is h
    want = plain.gated(x, wg, wu, act)
    g, u = x.double().cpu() @ wg.double().cpu().t(), x.double().cpu() @ wu.double().cpu().t()
    _, eu, ev, _ = gated_slack(x, wg, wu, act)
    value = plain.activation(g, act)[0]
    bound = ev * (u.abs() + eu) + value.abs() * eu + (HALF_ULP[dtype] + 4 * U) * want.abs() + TINY[dtype]
    err = (h.double().cpu() - want).abs()
    assert (err <= bound).all(), (err / bound.clamp(min=1e-300)).max()
    assert untouched(h, hw)
    odd, oddw = window(torch.zeros(m, f), REALS[dtype], 1, extra=f % 2 + 2)
    fwt.gated(x, wg, wu, activation=act, out=odd)
    assert torch.equal(odd, h) and untouched(odd, oddw)
    assert torch.equal(fwt.gated(x, wg, wu, activation=act), h)


@pytest.mark.parametrize("m", [2, 20, 150])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gated_special_values(m, act):
    """A NaN in a row of x or of a weight spoils that row or column alone; far from zero the
    activation has its limits."""
    x, wg, wu, _ = gated_inputs(m, 64, 300, "bf16")
    x[:, 0] = 0
    clean = fwt.gated(x, wg, wu, activation=act)
    y = x.clone()
    y[1, 5] = NAN
    out = fwt.gated(y, wg, wu, activation=act)
    assert torch.isnan(out[1]).all()
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(out[keep], clean[keep])
    w2 = wu.clone()
    w2[17] = NAN
    out = fwt.gated(x, wg, w2, activation=act)
    assert torch.isnan(out[:, 17]).all() and torch.equal(out[:, 18:], clean[:, 18:])
    big = torch.full((m, 64), 100.0, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(300, 64, dtype=torch.bfloat16, device="cuda")
    assert (fwt.gated(big, -ones, ones, activation=act) == 0).all()
    assert (fwt.gated(big, ones, ones, activation=act) == 6400.0 * 6400.0).all()


BACKWARD = [
    (1, 8, 1, "bf16", "silu"), (1, 256, 1000, "bf16", "silu"), (3, 1, 5, "f16", "gelu"),
    (7, 130, 257, "f16", "relu"), (16, 512, 512, "bf16", "gelu"), (33, 1001, 531, "bf16", "silu"),
    (100, 64, 72, "f16", "silu"), (128, 128, 128, "bf16", "silu"), (130, 257, 700, "bf16", "gelu"),
    (517, 333, 401, "f16", "gelu"), (600, 1024, 900, "bf16", "silu"), (1025, 128, 260, "bf16", "relu"),
    (1, 1500, 300, "f16", "silu"), (2, 2048, 70, "bf16", "relu"), (5, 1001, 900, "bf16", "gelu"),
    (8, 260, 2057, "f16", "silu"), (9, 700, 520, "f16", "relu"),
    (40, 300, 1100, "bf16", "gelu"), (300, 1700, 400, "f16", "silu"), (250, 1200, 1000, "bf16", "silu"),
    (256, 1900, 800, "bf16", "silu"), (500, 2000, 700, "f16", "gelu"), (2000, 300, 500, "bf16", "silu"),
    (1500, 500, 700, "f16", "silu"), (1400, 640, 500, "bf16", "gelu"), (1800, 128, 128, "bf16", "silu"), (300, 72, 4900, "f16", "silu"), (70, 4900, 300, "bf16", "gelu"),
    (1500, 1303, 2105, "bf16", "silu"), (2307, 2500, 300, "f16", "gelu"),
]


def backward_bounds(grad, x, wg, wu, act, dtype):
    dg, du = plain.gated_parts(grad, x, wg, wu, act)
    eg, eu, ev, es = gated_slack(x, wg, wu, act)
    dh, xd, wgd, wud = (t.double().cpu().abs() for t in (grad, x, wg, wu))
    g, u = x.double().cpu() @ wg.double().cpu().t(), x.double().cpu() @ wu.double().cpu().t()
    slope = plain.activation(g, act)[1]
    half = HALF_ULP[dtype] + 8 * U
    edg = dh * (u.abs() * es + (slope.abs() + es) * eu) + half * dg.abs() + TINY[dtype]
    edu = dh * ev + half * du.abs() + TINY[dtype]
    edg, edu = edg * (1 + 2 * half), edu * (1 + 2 * half)
    want = plain.gated_backward(grad, x, wg, wu, act)
    m, f = grad.shape
    sums = (edg @ wgd + edu @ wud + 2 * f * 2 * U * (dg.abs() @ wgd + du.abs() @ wud),
            edg.t() @ xd + m * 2 * U * (dg.abs().t() @ xd),
            edu.t() @ xd + m * 2 * U * (du.abs().t() @ xd))
    return want, [s * 1.01 + HALF_ULP[dtype] * w.abs() + TINY[dtype] for s, w in zip(sums, want)]


@pytest.mark.parametrize("m,d,f,dtype,act", BACKWARD)
def test_gated_backward(m, d, f, dtype, act):
    x, wg, wu, grad = gated_inputs(m, d, f, dtype, extra=1)
    outs = [window(torch.zeros(s), REALS[dtype], 8, extra=1) for s in ((m, d), (f, d), (f, d))]
    got = fwt.gated_backward(grad, x, wg, wu, activation=act, out=tuple(o[0] for o in outs))
    want, bounds = backward_bounds(grad, x, wg, wu, act, dtype)
    for name, a, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        err = (a.double().cpu() - w).abs()
        assert (err <= b).all(), (name, (err / b.clamp(min=1e-300)).max())
    assert all(untouched(*o) for o in outs)
    again = fwt.gated_backward(grad, x, wg, wu, activation=act)
    assert all(torch.equal(a, b) for a, b in zip(again, got))
    only_x = fwt.gated_backward(grad, x, wg, wu, activation=act, want=("x",))
    assert torch.equal(only_x[0], got[0]) and only_x[1] is None and only_x[2] is None
    only_w = fwt.gated_backward(grad, x, wg, wu, activation=act, want=("w",))
    assert only_w[0] is None and torch.equal(only_w[1], got[1]) and torch.equal(only_w[2], got[2])
    odd = [window(torch.zeros(s), REALS[dtype], 1, extra=s[1] % 2 + 2) for s in ((m, d), (f, d), (f, d))]
    fwt.gated_backward(grad, x, wg, wu, activation=act, out=tuple(o[0] for o in odd))
    assert all(torch.equal(o[0], g) and untouched(*o) for o, g in zip(odd, got))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward_against_differences(act):
    """Directional derivatives of the exact loss <grad, h> by central differences."""
    m, d, f = 40, 96, 130
    x, wg, wu, grad = gated_inputs(m, d, f, "bf16")
    got = [t.double().cpu() for t in fwt.gated_backward(grad, x, wg, wu, activation=act)]
    base = [t.double().cpu() for t in (x, wg, wu)]
    dh = grad.double().cpu()
    for i in range(3):
        v = torch.randn(base[i].shape, generator=gen(50 + i), dtype=torch.float64)
        step = 1e-4
        sides = []
        for sign in (1, -1):
            t = list(base)
            t[i] = t[i] + sign * step * v
            sides.append((dh * plain.gated(*t, act)).sum())
        slope = (sides[0] - sides[1]) / (2 * step)
        # two roundings to 8 significant bits (the operand dg or du, and the output), each
        # uniform within 2^-8, so at most 2^-8 sqrt(2 / 3) together: five standard deviations
        tolerance = 5 * 2.0 ** -8 * got[i].norm() + 1e-6
        assert abs((got[i] * v).sum() - slope) <= tolerance


def test_gated_over_nothing():
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, hw = window(torch.ones(5, 9), torch.bfloat16, 8)
    fwt.gated(empty(5, 0), empty(9, 0), empty(9, 0), out=h)
    assert (h == 0).all() and untouched(h, hw)
    assert fwt.gated(empty(0, 16), empty(9, 16), empty(9, 16)).shape == (0, 9)
    w = torch.ones(9, 16, dtype=torch.bfloat16, device="cuda")
    dx, dwg, dwu = fwt.gated_backward(empty(0, 9), empty(0, 16), w, w)
    assert dx.shape == (0, 16) and (dwg == 0).all() and (dwu == 0).all()
    x = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    dx, dwg, dwu = fwt.gated_backward(empty(4, 0), x, empty(0, 16), empty(0, 16))
    assert (dx == 0).all() and dwg.shape == (0, 16)
    dx, dwg, dwu = fwt.gated_backward(torch.ones(4, 9, dtype=torch.bfloat16, device="cuda"),
                                      empty(4, 0), empty(9, 0), empty(9, 0))
    assert dx.shape == (4, 0) and dwg.shape == (9, 0)


# ---- streams, graphs ---------------------------------------------------------------

def chain(x, wg, wu, q_down, s_down, stream=None):
    h = fwt.gated(x, wg, wu, stream=stream)
    q, s = fwt.quantize_blocks(h, rotate=7, stream=stream)
    return h, q, s, fwt.matmul_blocks(q, s, q_down, s_down, stream=stream)


@pytest.mark.parametrize("m", [1, 24, 200])
def test_streams_and_graph_capture(m):
    x, wg, wu, grad = gated_inputs(m, 256, 640, "bf16")
    down = torch.randn(256, 640, generator=gen(3)).to(torch.bfloat16).cuda()
    qd, sd = fwt.quantize_blocks(down, rotate=7, lines=128)
    want = chain(x, wg, wu, qd, sd)[3].clone()
    want_grads = [t.clone() for t in fwt.gated_backward(grad, x, wg, wu)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = chain(x, wg, wu, qd, sd, stream=side)
    grads = fwt.gated_backward(grad, x, wg, wu, stream=side)
    side.synchronize()
    assert torch.equal(kept[3], want) and all(torch.equal(a, b) for a, b in zip(grads, want_grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain(x, wg, wu, qd, sd)
        grads = fwt.gated_backward(grad, x, wg, wu)
    x2 = x.clone()
    x.copy_(x2 * 0.5)
    graph.replay()
    torch.cuda.synchronize()
    half = chain(x, wg, wu, qd, sd)[3]
    assert torch.equal(kept[3], half) and not torch.equal(kept[3], want)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept[3], want) and all(torch.equal(a, b) for a, b in zip(grads, want_grads))
    assert fwt.device_status() == fwt.FWT_OK


@pytest.mark.parametrize("raw", [False, True])
def test_allocations_belong_to_the_calls_stream(raw):
    """Memory that a call on another stream allocates is not the current stream's to hand on:
    a temporary of a chain on `side` may still be read there when its tensor is gone."""
    m, d, f = 1024, 512, 4096  # 8 MB of h: blocks that the allocator keeps and hands on again
    x, wg, wu, grad = gated_inputs(m, d, f, "bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = side.cuda_stream if raw else side

    def outputs():
        h = fwt.gated(x, wg, wu, stream=stream)
        codes, scale = fwt.quantize_blocks(h, rotate=7, lines=128, stream=stream)
        c = fwt.matmul_blocks(codes, fwt.quantize_blocks(h, stream=stream)[1], codes, scale,
                              stream=stream)
        return [h, codes, c, *fwt.gated_backward(grad, x, wg, wu, stream=stream)]

    made = outputs()
    side.synchronize()
    freed = [(t.data_ptr(), t.numel() * t.element_size()) for t in made]
    sizes = sorted({size for _, size in freed})
    del made
    taken = []  # as many blocks of each size on the current stream as were freed, and more
    for size in sizes:
        taken += [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(len(freed) + 1)]
    for t in taken:
        for at, size in freed:
            assert t.data_ptr() >= at + size or at >= t.data_ptr() + t.numel()
    assert fwt.device_status() == fwt.FWT_OK


def test_the_default_stream_by_its_handle():
    x, wg, wu, grad = gated_inputs(24, 256, 640, "f16")
    want = [fwt.gated(x, wg, wu), *fwt.gated_backward(grad, x, wg, wu)]
    torch.cuda.synchronize()
    for handle in (0, 1):
        got = [fwt.gated(x, wg, wu, stream=handle), *fwt.gated_backward(grad, x, wg, wu, stream=handle)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fwt.device_status() == fwt.FWT_OK
