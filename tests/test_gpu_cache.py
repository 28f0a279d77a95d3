"""Cache operators on the GPU against 64 bits: written, read back, attended to."""
import math

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import (E4M3_OF, HALF_ULP, REALS, TINY, Problem, check_attention, quantised, raw, turned)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fresh():
    torch.manual_seed(0)
    yield
    assert fwt.device_status() == fwt.FWT_OK


def rows(tokens, heads, dim, dtype, spread=1.0):
    x = torch.randn(tokens, heads, dim) * torch.exp(spread * torch.randn(heads, dim))
    return x.to(REALS[dtype]).cuda()


# ---- written ---------------------------------------------------------------------------

def check_held(pr, b, name, x, r, first):
    """Sequence b's last tokens are x (n, heads, dim), rotated and cut."""
    values, there = pr.held(name, b)
    values, there = values[first:], there[first:]
    code, byte, y = quantised(x.cpu(), r)
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(byte == 255, math.nan, torch.exp2(byte.double() - 127))[..., None]
    # fp32: r sums, the norm and its product; a code on the border may go either way, and a scale by 2
    fine = 2.0 ** -24 * (r + 2) * y.abs().amax(-1, keepdim=True) * 2
    # half a step of e4m3: 2^-4 of the value, at least 2^-10 of the scale (twice that for a scale by two)
    room = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * scale) + fine
    border = (top / scale / 448 - 1).abs() < 2.0 ** -20
    border |= (top / scale / 224 - 1).abs() < 2.0 ** -20
    room = torch.where(border, torch.maximum(room, 2.0 ** -9 * scale), room)
    nan = (byte == 255)[..., None].expand_as(values)
    assert torch.equal(torch.isnan(values[there]), nan[there])
    off = torch.where(nan, 0.0, (values - y).abs())
    assert (off <= torch.where(nan, 1.0, room))[there].all(), (off / room).max()
    # as the codes of the rounded value, for nearly all
    same = (values == torch.where(nan, 0.0, code * scale)) | nan
    assert same[there].double().mean() > 0.999 if same[there].numel() > 2000 else True


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("news,lens,heads,dim,page,r", [
    ([1], [1], 1, 64, 16, 6), ([1], [1], 1, 128, 16, 7), ([5], [5], 3, 64, 16, 0), ([17, 0, 1, 40], [17, 3, 90, 47], 2, 128, 16, 7),
    ([3, 4], [100, 4], 5, 64, 48, 4), ([130], [333], 8, 128, 64, 5), ([33, 200, 9], [64, 201, 4000], 7, 128, 128, 3),
    ([1] * 300, [(37 * i) % 90 + 1 for i in range(300)], 2, 64, 32, 6), ([9] * 5, [200] * 5, 3, 128, 1008, 1)])
def test_append(news, lens, heads, dim, page, r, dtype):
    pr = Problem(news, lens, heads, dim, page, tail=3, codes=False)
    before = [raw(t).clone() for t in pr.cache]
    k, v = (rows(pr.tokens, heads, dim, dtype) for _ in range(2))
    assert fwt.cache_append(k, v, *pr.places(), rotate=r) is pr.cache
    touched = torch.zeros(pr.pages, page, dtype=torch.bool)
    for b, n in enumerate(news):
        at = torch.arange(lens[b] - n, lens[b])
        touched[pr.table[b].cpu().long()[at // page], at % page] = True
        s = slice(int(pr.starts[b]), int(pr.starts[b + 1]))
        check_held(pr, b, "k", k[s], r, lens[b] - n)
        check_held(pr, b, "v", v[s], r, lens[b] - n)
    for old, new in zip(before, pr.cache):  # the rest of the cache is as it was
        keep = ~touched[:, None].expand(-1, heads, -1).cuda()
        assert torch.equal(old[keep], raw(new)[keep])


def test_append_scales_at_their_borders():
    """Largest magnitudes next to 448 times a power of two, the range's ends, zeros and what is not a
    number, without a rotation (so that y is x): the scale is the least that holds them."""
    tops = torch.tensor([448.0, 448.0 * (1 + 2.0 ** -23), 447.0, 1.75, 1.0, 0.0, -0.0, 3e38, 2.0 ** -118, 448 * 2.0 ** -126,
                         449 * 2.0 ** -126, 2.0 ** -126, 1e-40, 2.0 ** -149, math.inf, -math.inf, math.nan])
    n = len(tops)
    pr = Problem([n], [n], 1, 64, 16, codes=False)
    x = torch.zeros(n, 1, 64)
    x[:, 0, 5], x[:, 0, 60] = tops, tops / 3
    fwt.cache_append(x.cuda(), -x.cuda(), *pr.places(), rotate=0)
    code, byte, _ = quantised(x, 0)
    for name, sign in (("k", 1.0), ("v", -1.0)):
        page = pr.table[0].cpu().long()[torch.arange(n) // 16]
        got = raw(getattr(pr.cache, name + "_scale")).cpu()[page, :, torch.arange(n) % 16]
        assert torch.equal(got.long(), byte)
        codes = E4M3_OF[raw(getattr(pr.cache, name)).cpu()[page, :, torch.arange(n) % 16].long()]
        assert torch.equal(codes, sign * code + 0.0)


def test_append_large_values_do_not_overflow_in_the_rotation():
    """128 values of 2^120: their sum passes fp32 on the way, the normalised one does not."""
    pr = Problem([2], [2], 1, 128, 16, codes=False)
    x = torch.full((2, 1, 128), 2.0 ** 121)
    x[1, 0, 7] = math.nan
    fwt.cache_append(x.bfloat16().cuda(), x.bfloat16().cuda(), *pr.places())
    check_held(pr, 0, "k", x, 7, 0)


def test_append_leaves_out_what_has_no_place():
    """Pages that are none, sequences shorter than their new tokens, lengths beyond the table and below
    zero, starts beyond the rows."""
    pr = Problem([4, 20, 5, 5, 6], [40, 20, 5, 5, 6], 2, 64, 16, codes=False, most_pages=3)
    pr.table[0, 2] = pr.pages          # one past the last page
    pr.table[1, 0] = -5
    pr.table[2, 0] = 2 ** 31 - 1
    pr.lengths[3] = -7                  # nothing
    pr.lengths[4] = 1 << 30             # as the table's 48 tokens
    pr.table[4, 1:] = torch.tensor([pr.pages - 1, pr.pages - 2])
    pr.starts[5] = 1000                 # as the packed rows' 40
    k, v = (rows(pr.tokens, 2, 64, "bf16") for _ in range(2))
    before = [raw(t).clone() for t in pr.cache]
    fwt.cache_append(k, v, *pr.places())
    touched = torch.zeros(pr.pages, 16, dtype=torch.bool)
    table = pr.table.cpu().long()
    touched[table[0, 1], 4:8] = False
    touched[table[1, 1], :4] = True     # tokens 16 .. 19 of sequence 1
    touched[table[4, 2], 10:] = True    # tokens 42 .. 47 of sequence 4
    # sequence 0: positions 36 .. 39, all in the page that is none
    for old, new in zip(before, pr.cache):
        same = (old == raw(new)).reshape(pr.pages, 2, 16, -1).all(-1).all(1).cpu()
        assert same[~touched].all()
        assert not same[touched].any()
    check_held(pr, 1, "k", k[8:24][-4:], 6, 16)


def test_append_takes_windows_and_pools():
    """Keys and values inside a fused projection, heads outside tokens, a layer of a pool of pages."""
    tokens, heads, dim, page, pages = 50, 3, 128, 32, 6
    pool = torch.zeros(pages, 2, 2, heads * page * dim, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, 2, 2, heads * page, dtype=torch.uint8, device="cuda")
    pr = Problem([tokens], [tokens], heads, dim, page, codes=False)
    cache = fwt.Cache(*(t[:, 1, o].view(pages, heads, page, *(() if s else (dim,))).view(
        torch.float8_e8m0fnu if s else torch.float8_e4m3fn) for o in range(2) for s, t in ((0, pool), (1, scales))))
    qkv = rows(tokens, 5 * heads, dim, "bf16")
    k = qkv[:, heads:2 * heads]
    v = rows(heads, tokens, dim, "bf16").transpose(0, 1)
    want = fwt.cache_append(k.contiguous(), v.contiguous(), *pr.places())
    pr.table.clamp_(max=pages - 1)
    fwt.cache_append(k, v, cache, *pr.places()[1:])
    at = torch.arange(tokens, device="cuda")
    for a, b in zip(cache, want):
        page_of = pr.table[0][at // page].long()
        assert torch.equal(raw(a)[page_of, :, at % page], raw(b)[page_of, :, at % page])
    assert pool[:, 0].count_nonzero() == 0 and scales[:, 0].count_nonzero() == 0
    back = torch.full((tokens, 2, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fwt.cache_read(cache, *pr.places()[1:], tokens, out=(back[:, 0], back[:, 1]))
    for x, y in zip(got, fwt.cache_read(*pr.places(), tokens)):
        assert torch.equal(x, y)


# ---- read back -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("news,lens,heads,dim,page,r", [
    ([1], [1], 1, 64, 16, 6), ([1], [1], 1, 128, 16, 7), ([17, 0, 1, 40], [17, 3, 90, 47], 2, 128, 16, 7),
    ([3, 4], [100, 4], 5, 64, 48, 4), ([130], [333], 8, 128, 64, 0), ([1] * 300, [(37 * i) % 90 + 1 for i in range(300)], 2, 64, 32, 5),
    ([20, 6], [10, 3], 2, 128, 32, 2)])
def test_read(news, lens, heads, dim, page, r, dtype):
    pr = Problem(news, lens, heads, dim, page, tail=4)
    if len(news) == 2:
        pr.table[1, 0] = -3 if news[0] == 20 else pr.pages + 5
    out = tuple(torch.full((pr.tokens, heads, dim), 9.0, dtype=REALS[dtype], device="cuda") for _ in range(2))
    got = fwt.cache_read(*pr.places(), pr.tokens, rotate=r, out=out)
    for name, x in zip("kv", got):
        assert (x[sum(news):] == 9).all()
        for b, n in enumerate(news):
            values, there = pr.held(name, b)
            values = torch.where(there[:, None, None], values, 0.0)
            pad = torch.zeros(max(0, n - lens[b]), heads, dim, dtype=torch.float64)
            y = turned(torch.cat([pad, values])[-n:] if n else pad, r)
            # sums of codes are exact to 2^-24 of their largest a bit; the norm and its product
            room = HALF_ULP[dtype] * y.abs() + TINY[dtype] + 2.0 ** -24 * (
                (r + 2) * y.abs().amax(-1, keepdim=True) * 2 ** (r / 2))
            off = (x[int(pr.starts[b]):int(pr.starts[b]) + n].double().cpu() - y).abs()
            assert (off <= room * (1 + 2.0 ** -10)).all()


def test_what_is_not_finite_comes_back_so():
    pr = Problem([3], [3], 2, 64, 16, codes=False)
    k, v = (rows(3, 2, 64, "f32") for _ in range(2))
    k[1, 0, 3], v[2, 1, 63] = math.inf, math.nan
    fwt.cache_append(k, v, *pr.places())
    a, b = fwt.cache_read(*pr.places(), 3, dtype=torch.float32)
    assert torch.isnan(a[1, 0]).all() and torch.isnan(b[2, 1]).all()
    assert torch.isfinite(a).sum() == torch.isfinite(b).sum() == 5 * 64


# ---- attended to -----------------------------------------------------------------------

SHAPES = [
    # news, lens, heads, group, dim, page
    ([1], [1], 1, 1, 64, 16), ([1], [1], 1, 1, 128, 16), ([1], [2], 2, 4, 128, 16), ([1], [16], 1, 8, 64, 16),
    ([1], [17], 1, 3, 128, 16), ([1], [33], 2, 1, 64, 32), ([1], [127], 3, 5, 128, 48), ([1], [129], 1, 16, 128, 16),
    ([1], [257], 2, 8, 64, 64), ([1], [1000], 2, 4, 128, 64), ([1], [4099], 2, 4, 128, 16), ([1], [5000], 1, 1, 64, 16),
    ([1, 1, 1], [70, 1, 700], 2, 4, 128, 16), ([1] * 40, [13 * i + 1 for i in range(40)], 2, 2, 64, 16),
    ([5, 5, 5], [5, 300, 77], 2, 2, 64, 16), ([2], [50], 4, 3, 128, 32), ([7, 0, 1, 3], [7, 20, 400, 45], 2, 8, 128, 16),
    ([31], [31], 2, 1, 128, 16), ([33], [100], 1, 1, 64, 16), ([64], [64], 1, 2, 128, 16), ([100, 3], [100, 200], 2, 3, 64, 48),
    ([129], [129], 1, 1, 128, 64), ([200], [900], 2, 4, 128, 64), ([255, 257, 1], [300, 257, 333], 1, 2, 64, 128),
    ([513], [513], 2, 1, 128, 128), ([300], [2000], 1, 5, 64, 16),
]


def queries(pr, group, dtype):
    return (torch.randn(pr.tokens, pr.heads * group, pr.dim) * 0.3).to(REALS[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("news,lens,heads,group,dim,page", SHAPES)
def test_attention(news, lens, heads, group, dim, page, dtype):
    pr = Problem(news, lens, heads, dim, page, tail=2, seed=len(news) + lens[0])
    q = queries(pr, group, dtype)
    r = [0, 4, 6 if dim == 64 else 7][sum(lens) % 3]
    out = torch.full_like(q, 5.0)
    got = fwt.cache_attention(q, *pr.places(), rotate=r, out=out)
    assert got is out and (out[sum(news):] == 5).all()
    check_attention(got, pr, q, r, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 17, 100, 1 << 40])
@pytest.mark.parametrize("news,lens,group,dim", [([1, 1], [300, 5], 4, 128), ([20, 3], [50, 222], 3, 64), ([70], [400], 2, 128),
                                                 ([300, 9], [600, 9], 1, 64)])
def test_masks(news, lens, group, dim, window, causal):
    pr = Problem(news, lens, 2, dim, 16, seed=3)
    q = queries(pr, group, "f16")
    got = fwt.cache_attention(q, *pr.places(), causal=causal, window=window)
    check_attention(got, pr, q, 6 if dim == 64 else 7, "f16", causal=causal, window=window)


@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128)])
@pytest.mark.parametrize("longest", [0, 500])
def test_rows_that_see_nothing_are_zero(group, dim, longest):
    """Empty sequences, more new tokens than the cache has, pages that are none, lengths out of range."""
    pr = Problem([3, 30, 5, 4, 6, 0, 2], [3, 10, 5, 70, 6, 0, 40], 2, dim, 16, most_pages=5, seed=4)
    pr.lengths[0] = 0
    pr.lengths[4] = -3
    pr.table[2, 0] = pr.pages
    pr.table[3, 1] = -1
    pr.table[3, 3] = 2 ** 31 - 1
    pr.lengths[6] = 2 ** 31 - 1         # as the table's 80 tokens, most of them without a page
    q = queries(pr, group, "bf16")
    got = fwt.cache_attention(q, *pr.places(), longest=longest)
    assert (got[:3] == 0).all() and (got[3:23] == 0).all() and (got[33:38] == 0).all()
    check_attention(got, pr, q, 6 if dim == 64 else 7, "bf16")


@pytest.mark.parametrize("news,lens,group,window", [([1], [300], 4, 0), ([40], [300], 4, 0), ([40], [300], 4, 25),
                                                    ([400], [700], 1, 0), ([400], [700], 1, 90)])
def test_what_is_not_a_number_goes_where_it_is_seen(news, lens, group, window):
    """Keys and values of a NaN scale: the rows that see them are NaN, the others as if there were none."""
    pr = Problem(news, lens, 2, 128, 32, seed=5)
    page, slot = pr.table.cpu().long(), None
    for name, head, token in (("k", 0, lens[0] - 1), ("v", 1, lens[0] - news[0] // 2 - 1), ("v", 0, lens[0] - news[0] // 4 - 1)):
        raw(getattr(pr.cache, name + "_scale"))[page[0, token // 32], head, token % 32] = 255
    if window:
        raw(pr.cache.v_scale)[page[0, 100 // 32], 0, 100 % 32] = 255  # before every window
    q = queries(pr, group, "f16")
    got = fwt.cache_attention(q, *pr.places(), window=window)
    check_attention(got, pr, q, 7, "f16", window=window)
    q[news[0] // 2, 1, 3] = math.inf   # a query's own row alone
    again = fwt.cache_attention(q, *pr.places(), window=window)
    assert torch.isnan(again[news[0] // 2, 1]).all()
    again[news[0] // 2, 1] = got[news[0] // 2, 1]
    assert torch.equal(again.isnan(), got.isnan()) and torch.equal(again.nan_to_num(), got.nan_to_num())


@pytest.mark.parametrize("new,length", [(1, 700), (70, 700), (300, 700)])
def test_scales_far_apart(new, length):
    """Values and keys whose scales lie many powers of two apart, in an order that makes the largest
    so far rise again and again; large and tiny queries."""
    pr = Problem([new], [length], 2, 128, 16, seed=6)
    table = pr.table[0].cpu().long()
    at = torch.arange(length)
    for name, low, high in (("k", 95, 118), ("v", 90, 160)):
        t = raw(getattr(pr.cache, name + "_scale"))
        byte = (low + (high - low) * at // length + torch.randint(-3, 4, (length,))).to(torch.uint8).cuda()
        t[table[at // 16].cuda(), :, (at % 16).cuda()] = byte[:, None].expand(-1, 2)
    for factor in (1.0, 2.0 ** -60, 2.0 ** 9):
        q = (queries(pr, 2, "bf16").float() * factor).bfloat16()
        check_attention(fwt.cache_attention(q, *pr.places()), pr, q, 7, "bf16")


def test_large_scores():
    """Scores of hundreds: one key has all the weight, and the maximum moves as keys go by."""
    pr = Problem([3], [900], 1, 128, 16, seed=7)
    q = (queries(pr, 4, "f16").float() * 40).half()
    check_attention(fwt.cache_attention(q, *pr.places(), rotate=0), pr, q, 0, "f16")


@pytest.mark.parametrize("longest", [1, 3, 9, 40, 400])
def test_longest_changes_nothing_but_the_way(longest):
    pr = Problem([1, 40, 3, 400], [300, 100, 3, 700], 2, 64, 16, seed=8)
    q = queries(pr, 3, "f16")
    check_attention(fwt.cache_attention(q, *pr.places(), longest=longest, rotate=0), pr, q, 0, "f16")


def test_many_sequences_and_pages_far_away():
    """More sequences than a CTA has threads, several without rows; a cache of over 4 GB whose last pages
    lie beyond 32-bit offsets."""
    n = 700
    pr = Problem([(i % 3) for i in range(n)], [(7 * i) % 50 + 2 for i in range(n)], 1, 64, 16, seed=9)
    q = queries(pr, 2, "bf16")
    check_attention(fwt.cache_attention(q, *pr.places()), pr, q, 6, "bf16")
    near = Problem([3, 1], [40, 90], 2, 128, 64, seed=10)
    pages = (9 << 29) // (2 * 64 * 128)
    far = fwt.new_cache(pages, 64, 2, 128)
    moved = near.table.clone()
    moved[near.table >= 0] += pages - near.pages
    for a, b in zip(far, near.cache):
        raw(a)[pages - near.pages:] = raw(b)
    k, v = (rows(4, 2, 128, "bf16") for _ in range(2))
    for cache, table in ((near.cache, near.table), (far, moved)):
        fwt.cache_append(k, v, cache, table, near.starts, near.lengths)
    for a, b in zip(far, near.cache):
        assert torch.equal(raw(a)[pages - near.pages:], raw(b))
    q = queries(near, 2, "bf16")
    want = fwt.cache_attention(q, *near.places())
    assert torch.equal(fwt.cache_attention(q, far, moved, near.starts, near.lengths), want)
    got = fwt.cache_read(far, moved, near.starts, near.lengths, 4)
    for a, b in zip(got, fwt.cache_read(*near.places(), 4)):
        assert torch.equal(a, b)


def test_strides_streams_graphs_and_workspaces():
    pr = Problem([1, 30], [200, 333], 2, 64, 16, seed=11)
    fused = torch.randn(pr.tokens, 10, 64, device="cuda").half()
    q = fused[:, 2:8]
    want = fwt.cache_attention(q.contiguous(), *pr.places())
    wide = torch.zeros(6, pr.tokens, 72, device="cuda").half()
    out = wide[:, :, :64].transpose(0, 1)
    assert torch.equal(fwt.cache_attention(q, *pr.places(), out=out), want)
    assert (wide[:, :, 64:] == 0).all()
    # out beside q in one tensor
    fwt.cache_attention(fused[:, :3].repeat(1, 2, 1), *pr.places())
    both = torch.cat([q, torch.zeros_like(q)], 1)
    fwt.cache_attention(both[:, :6], *pr.places(), out=both[:, 6:])
    assert torch.equal(both[:, 6:], want)
    # another stream, and results that repeat bit for bit
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fwt.cache_attention(q, *pr.places(), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # a graph that is replayed as sequences grow, with its workspace shared by a second graph
    size = fwt.fwt_cache_attention_workspace_bytes(6, 2, 64, 16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(want) for _ in range(2)]
    table, starts, lengths = pr.table.clone(), pr.starts.clone(), pr.lengths.clone()
    graphs = []
    for out in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fwt.cache_attention(q, pr.cache, table, starts, lengths, out=out, workspace=ws)
    for step in range(3):
        lengths.copy_(pr.lengths - 40 * step)
        expected = fwt.cache_attention(q, pr.cache, table, starts, lengths)
        for graph, out in zip(graphs, outs):
            out.zero_()
            graph.replay()
        assert torch.equal(outs[0], expected) and torch.equal(outs[1], expected)


def test_refusals_on_tensors():
    pr = Problem([2], [40], 2, 64, 16)
    q = queries(pr, 2, "f16")
    c, table, starts, lengths = pr.places()
    for bad, error in ((dict(q=q.float()), TypeError), (dict(q=q[:, :3]), ValueError), (dict(q=q[..., :32]), ValueError),
                       (dict(q=q[0]), ValueError), (dict(table=table.long()), TypeError), (dict(starts=starts[:1]), ValueError),
                       (dict(lengths=lengths.cpu()), ValueError), (dict(table=table[0]), ValueError), (dict(out=q), fwt.FwtError),
                       (dict(out=q.bfloat16()), TypeError), (dict(window=-1), ValueError), (dict(rotate=7), ValueError),
                       (dict(workspace=torch.zeros(64, device="cuda")), fwt.FwtError), (dict(scale=math.inf), fwt.FwtError),
                       (dict(workspace=torch.zeros(64)), ValueError)):
        args = {"q": q, "cache": c, "table": table, "starts": starts, "lengths": lengths, **bad}
        with pytest.raises(error):
            fwt.cache_attention(**args)
    odd = torch.zeros(2 * 2 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(2, 2, 64)
    with pytest.raises(fwt.FwtError, match="k starts at 2 bytes past"):
        fwt.cache_append(odd, odd, c, table, starts, lengths)
    with pytest.raises(ValueError):
        fwt.cache_append(odd, odd[:1], c, table, starts, lengths)
    with pytest.raises(TypeError):
        fwt.cache_append(odd, odd.float(), c, table, starts, lengths)
    with pytest.raises(ValueError):
        fwt.cache_read(c, table, starts, lengths, 3, out=(odd, odd))


# ---- together --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_prompt_its_chunks_and_its_tokens(dtype):
    """Prompts in chunks, then token by token, two sequences at different places in one call: what
    attention gives is that of the values read back, at every step."""
    heads, group, dim, page = 2, 3, 128, 16
    pr = Problem([0, 0], [150, 90], heads, dim, page, codes=False, seed=12)
    tol = HALF_ULP[dtype]
    done = [0, 0]
    for news in ((70, 33), (64, 1), (1, 50), (1, 1), (14, 5)):
        tokens = sum(news)
        pr.starts = torch.tensor([0, news[0], tokens], dtype=torch.int32, device="cuda")
        done = [d + n for d, n in zip(done, news)]
        pr.lengths = torch.tensor(done, dtype=torch.int32, device="cuda")
        pr.tokens = tokens
        k, v = (rows(tokens, heads, dim, dtype, 0.3) for _ in range(2))
        q = rows(tokens, heads * group, dim, dtype, 0.3) * 0.5
        fwt.cache_append(k, v, *pr.places())
        got = fwt.cache_attention(q, *pr.places())
        check_attention(got, pr, q, 7, dtype)
        every = torch.tensor([0, done[0], sum(done)], dtype=torch.int32, device="cuda")
        kk, vv = fwt.cache_read(pr.cache, pr.table, every, pr.lengths, sum(done), dtype=torch.float32)
        row = 0
        for b in range(2):
            ks, vs = (x[int(every[b]):int(every[b + 1])].double() for x in (kk, vv))
            for i in range(news[b]):
                n = done[b] - news[b] + i + 1
                for h in range(heads * group):
                    w = torch.softmax(ks[:n, h // group] @ q[row, h].double() * dim ** -0.5, 0)
                    want = w @ vs[:n, h // group]
                    # the roundings that check_attention counts, and those of the values read back (2^-24)
                    room = 6 * (tol * want.norm() + 2.0 ** -11 * 4 * (w @ vs[:n, h // group].norm(dim=-1)))
                    assert (got[row, h].double() - want).norm() <= room
                row += 1
