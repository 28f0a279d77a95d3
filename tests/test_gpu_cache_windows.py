"""Windows of more than 2^30 tokens on sequences that are longer still (one page named again and again)."""
import math

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import E4M3_OF, Problem, check_attention, raw

pytestmark = pytest.mark.gpu
PAGE = 1 << 20
CODE_OF_ONE = 0x38


@pytest.mark.parametrize("window,first", [
    ((1 << 30) + 5 * PAGE + 3, 35 * PAGE - 3),   # in tokens, the first that is seen
    ((1 << 30) + 39 * PAGE + 1, PAGE - 1),
    (1 << 31, 0), (1 << 40, 0),
    ((1 << 30) - 7, 40 * PAGE + 7)])
@pytest.mark.parametrize("longest", [1, 300])
def test_long_windows(window, first, longest):
    """Keys that score 0 but for the last of four pages, which have all the weight that the window leaves them."""
    pages = 1024 + 40
    cache = fwt.new_cache(3, PAGE, 1, 64)
    gen = torch.Generator().manual_seed(3)
    raw(cache.k_scale).fill_(127)
    raw(cache.v_scale).fill_(127)
    values = torch.randint(0x20, 0x60, (3, 64), generator=gen).to(torch.uint8)
    raw(cache.v)[:] = 0x30
    for page in (1, 2):
        raw(cache.k)[page, 0, PAGE - 1, 0] = CODE_OF_ONE
        raw(cache.v)[page, 0, PAGE - 1] = values[page].cuda()
    table = torch.zeros(1, pages, dtype=torch.int32)
    table[0, 0], table[0, 34], table[0, 38], table[0, 41] = 1, 1, 2, 2
    marks = {PAGE - 1: 1, 35 * PAGE - 1: 1, 39 * PAGE - 1: 2, 42 * PAGE - 1: 2}
    length = pages * PAGE
    q = torch.zeros(1, 1, 64, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    args = (table.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
            torch.tensor([length], dtype=torch.int32, device="cuda"))
    got = fwt.cache_attention(q, cache, *args, rotate=0, scale=60 * math.log(2), window=window, longest=longest)
    assert first == max(0, length - window)
    seen = [p for at, p in marks.items() if at >= first]
    want = E4M3_OF[values[seen].long()].mean(0)
    # the other 2^30 keys weigh 2^-30 of one of these; roundings as elsewhere, 2^-11 each of p and the output
    off = (got[0, 0].double().cpu() - want).abs()
    assert (off <= 2.0 ** -10 * want + 2.0 ** -16).all(), off.max()


@pytest.mark.parametrize("longest", [1, 300])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 5, 1 << 30, (1 << 31) - 1, 1 << 50])
def test_positions_below_zero(window, causal, longest):
    """More new tokens than the cache has: the first stand before its first token and, causally, see nothing."""
    pr = Problem([20], [12], 2, 64, 16, seed=4)
    q = (torch.randn(20, 4, 64) * 0.3).half().cuda()
    got = fwt.cache_attention(q, *pr.places(), window=window, causal=causal, longest=longest)
    check_attention(got, pr, q, 6, "f16", window=window, causal=causal)
