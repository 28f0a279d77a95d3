"""matmul_blocks with scales whose products leave the range of fp32, and with the least."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import U, matmul_expected, operand

pytestmark = pytest.mark.gpu
SIZES = [(5, 300, 400), (30, 200, 1400), (60, 700, 300), (300, 400, 1500), (2307, 2500, 400)]


def scaled(m, n, k, lines, a_factors, b_factors):
    """Operands whose scales of block t are some power of two times a_factors[t % ..] and so on."""
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, lines, 2)
    sa = sa * torch.tensor(a_factors, device="cuda")[torch.arange(sa.shape[1]) % len(a_factors)]
    sb = sb * torch.tensor(b_factors, device="cuda")[torch.arange(sb.shape[1]) % len(b_factors)]
    return a, sa, b, sb


def check(a, sa, b, sb, lines, k, least=0.0):
    want, size = matmul_expected(a, sa, b, sb, lines)
    got = fwt.matmul_blocks(a, sa, b, sb, out_dtype=torch.float32).double().cpu()
    # (a sum times one scale and then the other: one rounding more than their product first)
    bound = (min(k, 128) + -(-k // 128) + 4) * 2 * U * size + 2.0 ** -24 * want.abs() + 2.0 ** -148 + least
    fits = want.abs() + bound < 3.4e38
    assert fits.any()
    err = (got - want).abs()
    assert (err[fits] <= bound[fits]).all(), (err[fits] / bound[fits]).max()
    over = want.abs() - bound > 3.41e38
    assert torch.isinf(got[over]).all()


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("lines", [1, 128])
def test_products_of_scales_beyond_fp32(m, n, k, lines):
    """A block of zeros, or of a few of the least codes, between scales of 2^70 each."""
    a, sa, b, sb = scaled(m, n, k, lines, [2.0 ** 70, 1.0], [2.0 ** 70, 1.0])
    for t in range(0, -(-k // 128), 2):
        b.view(torch.uint8)[:, 128 * t:128 * t + 128] = 0
        a.view(torch.uint8)[:, 128 * t:128 * t + 128] = 0
    check(a, sa, b, sb, lines, k)
    a.view(torch.uint8)[:, 3] = 1   # 2^-9
    b.view(torch.uint8)[::2, 3] = 1
    sb[:, 0] = 2.0 ** 66
    sa[:, 0] = 2.0 ** 68
    check(a, sa, b, sb, lines, k)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("lines", [1, 128])
@pytest.mark.parametrize("factors", [(2.0 ** -68, 2.0 ** -63), (2.0 ** 10, 2.0 ** -120), (2.0 ** 100, 2.0 ** -100)])
def test_products_of_scales_below_fp32(m, n, k, lines, factors):
    """The product of two scales is rounded to fp32: below 2^-126 to steps of 2^-149, which times a
    block's sum of at most 128 * 448^2 is off by 2^-125 at most."""
    small = factors[0] * factors[1] < 1
    check(*scaled(m, n, k, lines, [factors[0]], [factors[1]]), lines, k,
          least=-(-k // 128) * 128 * 448.0 ** 2 * 2.0 ** -150 if small else 0.0)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("lines", [1, 128])
def test_blocks_of_nothing_at_the_least_scale(m, n, k, lines):
    a, sa, b, sb = scaled(m, n, k, lines, [1.0], [1.0])
    want = fwt.matmul_blocks(a[:, 128:], sa[:, 1:], b[:, 128:], sb[:, 1:], out_dtype=torch.float32)
    a.view(torch.uint8)[:, :128] = 0
    sa[:, 0] = 2.0 ** -126
    full = fwt.matmul_blocks(a, sa, b, sb, out_dtype=torch.float32)
    check(a, sa, b, sb, lines, k)
    assert full.shape == want.shape
