"""Values next to either end of fp32's range: what is finite as a mean is so on the way."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import Problem, check_attention, raw

pytestmark = pytest.mark.gpu
# a few rows in one share and in several, and many rows in both
CALLS = [([1], [700], 4), ([1] * 300, [50] * 300, 2), ([3, 2], [500, 90], 4), ([70], [400], 2), ([300, 9], [700, 30], 1),
         ([300] * 9, [310] * 9, 1)]


def problem(news, lens, dim, seed):
    torch.manual_seed(seed)
    return Problem(news, lens, 2, dim, 16, seed=seed)


@pytest.mark.parametrize("rotate", [0, 3, None])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,lens,group", CALLS)
def test_large_values(news, lens, group, dim, rotate):
    """Values of up to 2^125: their mean is finite, their sum is not."""
    pr = problem(news, lens, dim, 33)
    t = raw(pr.cache.v_scale)
    t[t != 255] = 243
    # of one sign in part, so that sums grow
    codes = raw(pr.cache.v)
    even = codes[..., ::2]
    codes[..., ::2] = torch.where(even & 0x7f == 0x7f, even, (even & 0x7f | 0x40).clamp(max=0x7e))
    q = (torch.randn(pr.tokens, 2 * group, dim) * 0.1).bfloat16().cuda()
    got = fwt.cache_attention(q, *pr.places(), rotate=rotate)
    r = (6 if dim == 64 else 7) if rotate is None else rotate
    assert torch.isfinite(got).all()
    check_attention(got, pr, q, r, "bf16")


@pytest.mark.parametrize("byte", [1, 2, 20])
@pytest.mark.parametrize("news,lens,group", CALLS[:4])
def test_small_values(news, lens, group, byte):
    """The other end: values of 2^-126 and the like, in shares as in one piece."""
    pr = problem(news, lens, 128, 34)
    t = raw(pr.cache.v_scale)
    t[t != 255] = byte
    q = (torch.randn(pr.tokens, 2 * group, 128) * 0.1).bfloat16().cuda()
    check_attention(fwt.cache_attention(q, *pr.places()), pr, q, 7, "bf16")
