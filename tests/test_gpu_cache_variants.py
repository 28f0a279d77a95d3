"""Which kernel a call of the cache operators takes, by the plan log; scores' scales of any sign; shares
that end inside items; a call that starts while the previous one still runs."""
import os
import subprocess
import sys

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_plain import Problem, check_attention, raw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = """
import sys
sys.path.insert(0, "tests")
import torch, walsh_hadamard_transform_gb300 as fwt
from cache_plain import Problem
for news, group, longest in (([1, 1], 8, 0), ([2, 2], 8, 0), ([3, 3], 8, 0), ([1, 40], 1, 0), ([1, 40], 1, 4)):
    pr = Problem(news, [n + 20 for n in news], 2, 64, 16)
    q = torch.randn(pr.tokens, 2 * group, 64, device="cuda").half()
    fwt.cache_attention(q, *pr.places(), longest=longest)
k = torch.randn(pr.tokens, 2, 64, device="cuda")
fwt.cache_append(k, k, *pr.places())
fwt.cache_read(*pr.places(), pr.tokens)
torch.cuda.synchronize()
"""


def test_plan_log():
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env=dict(os.environ, FWT_LOG="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln[5:] for ln in r.stderr.splitlines() if ln.startswith("fwt: ")]
    rows = []
    for line in lines[:-2]:
        rows.append(int(line.split("rows=")[1].split()[0]))
    assert rows == [n for each in (8, 16, 256, 256, 8) for n in (each, each)], lines
    assert [line.startswith("cache_attention join") for line in lines[:-2]] == [False, True] * 5
    assert lines[-2].startswith("cache_append tokens=41 heads=2 dim=64") and lines[-1].startswith("cache_read tokens=41 ")


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 0.7])
@pytest.mark.parametrize("new,group", [(2, 3), (90, 3)])
def test_scales_of_scores(new, group, scale):
    pr = Problem([new], [200], 2, 128, 16, seed=21)
    q = (torch.randn(new, 2 * group, 128) * 0.2).half().cuda()
    got = fwt.cache_attention(q, *pr.places(), scale=scale)
    check_attention(got, pr, q, 7, "f16", scale=scale)


@pytest.mark.parametrize("news,lens,heads,group,dim", [
    ([1], [20000], 1, 1, 128),                # one item over all workers
    ([1] * 9, [4096] * 9, 3, 2, 64),          # shares and items end at different places
    ([130] * 3, [9000, 131, 4000], 2, 1, 128),
    ([40], [30000], 1, 8, 64)])
def test_items_over_many_workers(news, lens, heads, group, dim):
    pr = Problem(news, lens, heads, dim, 64, seed=22)
    q = (torch.randn(pr.tokens, heads * group, dim) * 0.2).half().cuda()
    got = fwt.cache_attention(q, *pr.places())
    assert torch.equal(got, fwt.cache_attention(q, *pr.places()))
    check_attention(got, pr, q, 6 if dim == 64 else 7, "f16")


@pytest.mark.parametrize("new", [1, 100])
def test_calls_after_one_another(new):
    """Written, attended to and read back in a chain over the same buffers, with and without early starts:
    the same bits."""
    results = []
    for mode in (1, 0):
        assert fwt.library().fwt_set_pdl(mode) == fwt.FWT_OK
        try:
            torch.manual_seed(5)
            pr = Problem([new, new], [1000, 700], 2, 128, 32, codes=False, seed=23)
            lengths = pr.lengths.clone()
            x = torch.randn(2 * new, 4, 128, device="cuda").bfloat16()
            for step in range(new, 1000, max(new, 97)):
                lengths.copy_(torch.tensor([step, min(step, 700)], device="cuda"))
                at = (pr.cache, pr.table, pr.starts, lengths)
                fwt.cache_append(x[:, :2], x[:, 2:], *at)
                k, v = fwt.cache_read(*at, 2 * new)
                x = (fwt.cache_attention(x, *at) + 0.1 * torch.cat([k, v], 1) + 0.5 * x).clamp(-3, 3)
            results.append([x] + [raw(t).clone() for t in pr.cache])
        finally:
            fwt.library().fwt_set_pdl(1)
    assert torch.isfinite(results[0][0]).all()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_thousands_of_sequences():
    """More sequences than one group of the plan holds: as in calls of a few thousand each.  (No item is cut:
    each has one step.)"""
    n = 9001
    pr = Problem([1 + i % 2 for i in range(n)], [2 + i % 30 for i in range(n)], 1, 64, 16, seed=24)
    q = (torch.randn(pr.tokens, 2, 64) * 0.3).bfloat16().cuda()
    for longest in (1, 40):  # both kernels
        got = fwt.cache_attention(q, *pr.places(), longest=longest)
        for b0 in range(0, n, 3001):
            b1 = min(n, b0 + 3001)
            first, last = int(pr.starts[b0]), int(pr.starts[b1])
            part = fwt.cache_attention(q[first:last], pr.cache, pr.table[b0:b1], pr.starts[b0:b1 + 1] - first,
                                       pr.lengths[b0:b1], longest=longest)
            assert torch.equal(part, got[first:last])
        few = Problem.__new__(Problem)
        few.__dict__.update(pr.__dict__, starts=pr.starts[:40], lengths=pr.lengths[:39], table=pr.table[:39])
        check_attention(got, few, q, 6, "bf16")
