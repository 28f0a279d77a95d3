"""Attention over many keys in one share: what a tensor core's sums lose to their rounding toward zero does not grow with
the number of keys."""
import math

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import E4M3_OF, HALF_ULP, REALS, raw, turned

pytestmark = pytest.mark.gpu
PAGE = 1024


def values(cache, name):
    """(heads, tokens of the pages in order, dim) in 64 bits on the GPU."""
    codes, byte = raw(getattr(cache, name)).long(), raw(getattr(cache, name + "_scale")).double()
    v = E4M3_OF.cuda()[codes] * torch.exp2(byte - 127)[..., None]
    return v.transpose(0, 1).reshape(v.shape[1], -1, v.shape[3])


def softmax_means(q, k, v, group, scale):
    """(heads * group, dim): the output of one row of queries (heads * group, dim) in 64 bits."""
    s = torch.einsum("hgd,hkd->hgk", q.double().view(k.shape[0], group, -1), k) * scale
    return torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), v).flatten(0, 1)


def attend(q, cache, pages, repeat, sequences, new, longest, rotate=0):
    """`new` rows, all q, of each of `sequences`, which see the cache's pages in order `repeat` times."""
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(sequences, repeat)
    starts = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * new
    lengths = torch.full((sequences,), pages * PAGE * repeat, dtype=torch.int32, device="cuda")
    return fwt.cache_attention(q[None].repeat(sequences * new, 1, 1), cache, table, starts, lengths, rotate=rotate,
                               causal=False, longest=longest)


# (sequences, new, group, longest): rows of 8 and 16, and many; about one item for each worker
WAYS = [(152, 1, 1, 1), (152, 2, 8, 2), (19, 1, 1, 300), (10, 150, 2, 300)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("repeat", [4, 64])
@pytest.mark.parametrize("sequences,new,group,longest", WAYS)
def test_long_sums_are_not_short(sequences, new, group, longest, repeat, dim):
    """65536 and a million keys, values of one sign."""
    pages, heads = 16, 8
    gen = torch.Generator().manual_seed(51)
    cache = fwt.new_cache(pages, PAGE, heads, dim)
    raw(cache.k)[:] = (torch.randint(0, 0x40, cache.k.shape, generator=gen)
                       + 128 * torch.randint(0, 2, cache.k.shape, generator=gen)).to(torch.uint8).cuda()
    raw(cache.v)[:] = torch.randint(0x38, 0x48, cache.v.shape, generator=gen).to(torch.uint8).cuda()
    raw(cache.k_scale).fill_(126)
    raw(cache.v_scale).fill_(127)
    q = (torch.randn(heads * group, dim, generator=gen) * 0.7).half().cuda()
    got = attend(q, cache, pages, repeat, sequences, new, longest).double()
    want = softmax_means(q, values(cache, "k"), values(cache, "v"), group, dim ** -0.5)
    # A sum of products is rounded toward zero, by at most 2^-23, each 8 keys.  Sums of 8192 keys, half as large
    # in the mean, are added up to nearest, and the last 8192 to the sum of all.  Other roundings are to nearest: of
    # their mean over the output's elements little is left.
    off = ((got - want) / want).mean().item()
    assert abs(off) <= 1.5 * 8192 / 8 * 2.0 ** -23 + 2.0 ** -15, off


@pytest.mark.parametrize("rotate", [0, None])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sequences,new,group,longest", WAYS)
def test_units_and_maxima_that_move_between_sums(sequences, new, group, longest, dtype, dim, rotate):
    """40960 keys whose scores spread out further and further and whose values' scales go up and down."""
    pages, heads = 40, 8
    n = pages * PAGE
    gen = torch.Generator().manual_seed(52)
    cache = fwt.new_cache(pages, PAGE, heads, dim)
    for t in (cache.k, cache.v):
        c = torch.randint(0, 254, t.shape, generator=gen)
        raw(t)[:] = torch.where(c < 0x7f, c, c + 1).to(torch.uint8).cuda() & 0xbf
    stretch = torch.arange(pages)
    raw(cache.k_scale)[:] = (124 + stretch // 16).to(torch.uint8).cuda()[:, None, None]
    raw(cache.v_scale)[:] = (127 + (stretch * 5) % 9 - 2 * (stretch // 8)).to(torch.uint8).cuda()[:, None, None]
    q = (torch.randn(heads * group, dim, generator=gen) * 8).to(REALS[dtype])
    r = 0 if rotate == 0 else (6 if dim == 64 else 7)
    qr = turned(q, r).cuda()
    k, v = values(cache, "k"), values(cache, "v")
    want = turned(softmax_means(qr, k, v, group, dim ** -0.5).cpu(), r).cuda()
    got = attend(q.cuda(), cache, pages, 1, sequences, new, longest, rotate=rotate).double()
    s = torch.einsum("hgd,hkd->hgk", qr.view(heads, group, -1), k) * dim ** -0.5
    w = torch.softmax(s, -1)
    # roundings of queries, which move scores (each of a score's products by 2^-11 at most and a third of that
    # in the root mean square; a mean over all keys), of p (independent) and of the output, and what is lost in
    # sums
    size = torch.sqrt(torch.einsum("hgd,hkd->hgk", qr.view(heads, group, -1) ** 2, k ** 2)) * dim ** -0.5
    spread = (v[:, None] - torch.einsum("hgk,hkd->hgd", w, v)[:, :, None]).norm(dim=-1)
    of_q = 2.0 ** -11 * torch.sqrt(torch.einsum("hgk,hgk,hgk->hg", w, size ** 2, spread ** 2))
    of_p = 2.0 ** -11 * torch.sqrt(torch.einsum("hgk,hkd->hg", w ** 2, v ** 2))
    of_sums = (1.5 * 2.0 ** -13 + 2.0 ** -18) * torch.einsum("hgk,hkd->hgd", w, v.abs()).norm(dim=-1)
    room = (of_q + 6 * of_p + of_sums).flatten() + HALF_ULP[dtype] * want.norm(dim=-1)
    off = (got - want).norm(dim=-1)
    assert (off <= room).all(), (off / room).max()


def check_weights(sequences, new, group, longest, gap, dim, repeat):
    """One key `gap` powers of two above all others, which are alike, and values of one: a sum of equal numbers is
    rounded the same way each time."""
    pages, heads = 4, 8
    cache = fwt.new_cache(pages + 1, PAGE, heads, dim)
    raw(cache.v)[:] = 0x38
    for t in (cache.k_scale, cache.v_scale):
        raw(t).fill_(127)
    raw(cache.k)[pages, :, 5, 0] = 0x38
    q = torch.zeros(sequences * new, heads * group, dim, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(sequences, repeat)
    table[:, 3] = pages
    starts = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * new
    lengths = torch.full((sequences,), pages * PAGE * repeat, dtype=torch.int32, device="cuda")
    got = fwt.cache_attention(q, cache, table, starts, lengths, rotate=0, causal=False, scale=gap * math.log(2),
                              longest=longest)
    # sums of p V as above, and half a unit of p and of the output; sums of p to nearest, by 2^-25 of them for each
    # of 1024 numbers at most (every eighth p of 8192 keys), and sums of such sums, of p and of p V
    room = 1.5 * 2.0 ** -13 + 2 * 2.0 ** -11 + (1024 + 2 * pages * PAGE * repeat / 8192) * 2.0 ** -25
    off = (got.double() - 1).abs().max().item()
    assert off <= room, off


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [0.3, 0.7, 1.1, 5.3, 25.5])
@pytest.mark.parametrize("sequences,new,group,longest", WAYS)
def test_weights_of_a_million_keys_add_up_to_one(sequences, new, group, longest, gap, dim):
    check_weights(sequences, new, group, longest, gap, dim, 256)


@pytest.mark.parametrize("gap", [0.3, 0.7, 1.1, 5.3])
@pytest.mark.parametrize("repeat", [4096, 16384])
def test_weights_of_many_millions_by_many_rows(gap, repeat):
    check_weights(19, 1, 1, 300, gap, 64, repeat)
