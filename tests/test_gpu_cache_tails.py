"""Attention whose weight lies in many small probabilities beside one key far above them: a first key
with a value of zeros, so that the others are all of the output."""
import math

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import E4M3_OF, HALF_ULP, REALS, Problem, raw

pytestmark = pytest.mark.gpu
CODE_OF_ONE = 0x38


def held(pr, name, length):
    """Codes of sequence 0's first tokens (length, heads, dim), in 64 bits."""
    at = torch.arange(length, device="cuda")
    return E4M3_OF[raw(getattr(pr.cache, name))[pr.table[0].long()[at // pr.page], :, at % pr.page].cpu().long()]


def sink(length, heads, dim, gap, seed=0):
    """A cache of one sequence whose first key scores `gap` powers of two above the others, which score 0, for a
    query of element 0 alone; a value of zeros for it, random ones for them; the output of each key head."""
    pr = Problem([1], [length], heads, dim, 64, seed=seed)
    raw(pr.cache.k).zero_()
    raw(pr.cache.k_scale).fill_(127)
    raw(pr.cache.v_scale).fill_(137)  # (so that float16 outputs are normal numbers)
    first = pr.table[0, 0].long()
    raw(pr.cache.k)[first, :, 0, 0] = CODE_OF_ONE
    raw(pr.cache.v)[first, :, 0] = 0
    small = 2.0 ** -gap
    return pr, small * held(pr, "v", length).sum(0) * 1024 / (1 + (length - 1) * small)


def attend(pr, sequences, new, group, longest, scale, dtype):
    """The output of `new` rows of each of `sequences`, all on the pages of the first, by key head."""
    q = torch.zeros(sequences * new, pr.heads * group, pr.dim)
    q[..., 0] = 1.0
    starts = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * new
    out = fwt.cache_attention(q.to(REALS[dtype]).cuda(), pr.cache, pr.table.repeat(sequences, 1), starts,
                              pr.lengths.repeat(sequences), rotate=0, scale=scale, causal=False, longest=longest)
    return out.double().cpu().view(-1, pr.heads, group, pr.dim)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [14.3, 20.3, 22.6, 24.6, 25.5, 26.4])
@pytest.mark.parametrize("sequences,new,group,length,longest", [
    (300, 1, 4, 4000, 1),        # few rows: items of 125 steps, two for each worker
    (300, 2, 7, 4000, 2),
    (40, 1, 4, 8000, 300),       # many rows: items of 63 steps, two for each worker
    (20, 300, 2, 6000, 300)])
def test_small_probabilities_count(sequences, new, group, length, longest, gap, dim, dtype):
    pr, want = sink(length, 8, dim, gap)
    got = attend(pr, sequences, new, group, longest, gap * math.log(2), dtype)
    # p of all keys but one is the same number, and so is its rounding to float16: half a unit, 2^-11, or 2^-36
    # of the largest where that is more.  Then the score (gap, in fp32, and once more in the exponent), the
    # sums, and the output's own rounding.
    room = max(2.0 ** -11, 2.0 ** (gap - 36)) + 2.0 ** -22 * gap + 2.0 ** -18 + HALF_ULP[dtype]
    off = ((got - want[:, None]).norm(dim=-1) / want[:, None].norm(dim=-1)).max().item()
    assert off <= room, (off, room)


@pytest.mark.parametrize("dim", [64, 128])
def test_the_way_that_longest_chooses_agrees(dim):
    """The same rows by both kernels, one sequence over all workers and several shares an item."""
    gap = 25.5
    pr, want = sink(9000, 3, dim, gap, seed=1)
    for longest in (1, 8, 9, 300):
        for sequences in (1, 5, 60):
            got = attend(pr, sequences, 2, 2, longest, gap * math.log(2), "bf16")
            off = (got - want[:, None]).norm(dim=-1) / want[:, None].norm(dim=-1)
            assert off.max().item() <= 2.0 ** (gap - 36) + 2.0 ** -22 * gap + 2.0 ** -18 + HALF_ULP["bf16"]


@pytest.mark.parametrize("rise", [3.0, 3.9, 4.1, 7.5])
def test_a_maximum_that_moves_step_by_step(rise):
    """Each 128 keys score `rise` powers of two above those before: the sums so far are brought to the new
    maximum, or probabilities pass it by as much as they may."""
    steps, heads, dim = 12, 8, 64
    n = 128 * steps
    pr = Problem([1], [n], heads, dim, 128, seed=2)
    raw(pr.cache.k).zero_()
    raw(pr.cache.k_scale).fill_(127)
    raw(pr.cache.v_scale).fill_(127)
    for s in range(steps):
        raw(pr.cache.k)[pr.table[0, s].long(), :, :, 0] = int((E4M3_OF[:127] == s).nonzero()[0])
    v = held(pr, "v", n)
    step = torch.arange(n) // 128
    w = torch.softmax(step.double() * rise * math.log(2), 0)
    each = torch.zeros(steps, heads, dim, dtype=torch.float64).index_add_(0, step, w[:, None, None] * v)
    want = each.sum(0)
    for longest in (1, 300):
        got = attend(pr, 40, 1, 1, longest, rise * math.log(2), "f16")[:, :, 0]
        # p is one number for the keys of a step: of their rounding, 2^-11 at most, each step's share of the output;
        # the output's own; fp32, scores of up to 83 among it
        room = 2.0 ** -11 * (each.norm(dim=-1).sum(0) + want.norm(dim=-1)) + 2.0 ** -16 * v.norm(dim=-1).amax()
        assert ((got - want).norm(dim=-1) <= room).all()
