"""Queries and scores next to the end of fp32's range: what is finite after the rotation is so on the way."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import Problem, check_attention, raw

pytestmark = pytest.mark.gpu
# a few rows in one share and in several, and many rows in both
CALLS = [([1], [700], 4), ([1] * 300, [50] * 300, 2), ([3, 2], [500, 90], 4), ([70], [400], 2), ([300, 9], [700, 30], 1)]


def problem(news, lens, dim, seed):
    torch.manual_seed(seed)
    return Problem(news, lens, 2, dim, 16, seed=seed)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,lens,group", CALLS)
def test_large_queries(news, lens, group, dim):
    """Rows whose sums of a whole head pass fp32 although the rotated row does not, over tiny keys."""
    pr = problem(news, lens, dim, 31)
    raw(pr.cache.k_scale)[raw(pr.cache.k_scale) != 255] = 1  # 2^-126
    q = torch.full((pr.tokens, 2 * group, dim), 2.0 ** 121)
    # every row a line of H times a factor, so that it has one large element after the rotation, or anything
    q[1::3] *= (1 - 2 * (torch.arange(dim) & 1)) * 2.0 ** 0.5
    q[2::3] = torch.randn(q[2::3].shape) * 2.0 ** 121
    q[0, 0] *= 2
    q = q.bfloat16().cuda()
    got = fwt.cache_attention(q, *pr.places())
    assert torch.isfinite(got).all()
    check_attention(got, pr, q, 6 if dim == 64 else 7, "bf16")
