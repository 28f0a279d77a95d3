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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("power", [20, 21, 22, 23, 24, 25, 30, 60, 120])
@pytest.mark.parametrize("new,longest", [(1, 1), (5, 5), (70, 70)])
def test_large_scores_of_large_queries(new, longest, power, dim):
    """Scores of up to 2^123 from queries of 2^120: one key's are far above all others, and a rounding of a score is
    many powers of two."""
    pr = problem([new], [300], dim, 32)
    signs = 1 - 2 * torch.randint(0, 2, (300, 2, dim))
    for t in range(300):
        page = pr.table[0, t // 16].long()
        raw(pr.cache.k)[page, :, t % 16] = (0x70 | (signs[t] < 0).to(torch.uint8) << 7).cuda()  # 128
    raw(pr.cache.k_scale).fill_(127 - 8)
    mine = torch.arange(new) * 3 + 11
    q = (signs[mine] * 1.7 * 2.0 ** power).bfloat16().cuda()
    got = fwt.cache_attention(q, *pr.places(), rotate=0, scale=0.07, causal=False, longest=longest).double().cpu()
    v, _ = pr.held("v", 0)
    assert ((got - v[mine]).abs() <= 2.0 ** -8 * v[mine].abs()).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("power", [0, 6, 12, *range(17, 30), 60, 110])
@pytest.mark.parametrize("news,lens,group", [([1], [700], 4), ([70, 3], [700, 300], 2)])
def test_outputs_lie_among_the_values(news, lens, group, power, dim):
    """Random scores of any size: an output is a mean of values, none of its elements beyond theirs."""
    pr = problem(news, lens, dim, 35)
    q = (torch.randn(pr.tokens, 2 * group, dim) * 2.0 ** power).bfloat16().cuda()
    for longest in (1, 300):
        got = fwt.cache_attention(q, *pr.places(), rotate=0, longest=longest).double().cpu()
        for b, n in enumerate(news):
            most = pr.held("v", b)[0].abs().amax(0).repeat_interleave(group, 0)
            rows = got[int(pr.starts[b]):int(pr.starts[b]) + n]
            assert (rows.abs() <= most * (1 + 2.0 ** -7)).all() and rows.norm(dim=-1).min() > 0
