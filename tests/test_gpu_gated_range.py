"""Gradients of the gated projections where the products of gradient and projection leave the
range of float16 while the gradients themselves do not."""
import math

import pytest
import torch

import feed_forward_plain as plain
import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import U, gated_slack, gen

pytestmark = pytest.mark.gpu


def make(rows, cols, seed, scale):
    t = torch.randn(rows, cols, generator=gen(seed), dtype=torch.float64) * scale
    wide = torch.zeros(rows, cols + -cols % 8, dtype=torch.float16)
    wide[:, :cols] = t.half()
    return wide.cuda()[:, :cols]


def inputs(size, m, d, f):
    """x, both weights and the gradient of h, whose size this is."""
    if size > 1:  # a small x and a large w_up: u is some 10, so |dg| passes 65504
        return (make(m, d, 1, 0.01), make(f, d, 2, 0.1 / math.sqrt(d)), make(f, d, 3, 32.0),
                make(m, f, 4, size))
    return (make(m, d, 1, 1.0), make(f, d, 2, 2 / math.sqrt(d)), make(f, d, 3, 1 / math.sqrt(d)),
            make(m, f, 4, size))


def check(x, wg, wu, grad, act, got):
    """As a product of operands that hold dg and du to 11 significant bits down to 2^-38 of a bound
    on them all, max |dh| |x| in a row times the longest row of the weights: that many bits lie
    between the top of float16 and its least step, less those that the bound may be too large by
    a rounding up to powers of two."""
    dg, du = plain.gated_parts(grad, x, wg, wu, act)
    _, eu, ev, es = gated_slack(x, wg, wu, act)
    dh, xd, wgd, wud = (t.double().cpu().abs() for t in (grad, x, wg, wu))
    slope = plain.activation(x.double().cpu() @ wg.double().cpu().t(), act)[1]
    u = (x.double().cpu() @ wu.double().cpu().t()).abs()
    m, f = grad.shape
    half = 2.0 ** -11 + 8 * U
    least = 0.0
    if m > 8:
        top = (dh.amax(1) * xd.norm(dim=1)).max() * max(wgd.norm(dim=1).max(), wud.norm(dim=1).max())
        least = (1.13 * top * 2.0 ** -38).item()
    else:
        half = 8 * U
    edg = dh * (u * es + (slope.abs() + es) * eu) + half * dg.abs() + least
    edu = dh * ev + half * du.abs() + least
    want = plain.gated_backward(grad, x, wg, wu, act)
    sums = (edg @ wgd + edu @ wud + 4 * f * U * (dg.abs() @ wgd + du.abs() @ wud),
            edg.t() @ xd + 2 * m * U * (dg.abs().t() @ xd),
            edu.t() @ xd + 2 * m * U * (du.abs().t() @ xd))
    for name, a, w, s in zip(("dx", "dw_gate", "dw_up"), got, want, sums):
        assert w.abs().max() < 65504
        bound = 1.01 * s + 2.0 ** -11 * w.abs() + 2.0 ** -25
        err = (a.double().cpu() - w).abs()
        assert (err <= bound).all(), (name, (err / bound).nan_to_num(nan=math.inf).max().item())


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("m,d,f", [(8, 1024, 64), (9, 1024, 64), (300, 1024, 64), (300, 96, 520),
                                   (9, 100, 1001), (700, 264, 130)])
@pytest.mark.parametrize("size", [1e4, 1e-6])
def test_gradients_beyond_the_range_of_float16(size, m, d, f, act):
    x, wg, wu, grad = inputs(size, m, d, f)
    if size > 1 and m > 8:
        assert plain.gated_parts(grad, x, wg, wu, act)[0].abs().max() > 65504 or d < 1000
    check(x, wg, wu, grad, act, fwt.gated_backward(grad, x, wg, wu, activation=act))


def test_a_gradient_that_is_not_finite_stays_in_its_row():
    x, wg, wu, grad = inputs(1e4, 40, 256, 130)
    clean = fwt.gated_backward(grad, x, wg, wu)
    bad = inputs(1e4, 40, 256, 130)[3]
    bad[3, 7] = float("inf")
    bad[5, 0] = float("nan")
    dx, dwg, dwu = fwt.gated_backward(bad, x, wg, wu)
    keep = [i for i in range(40) if i not in (3, 5)]
    assert torch.equal(dx[keep], clean[0][keep]) and not torch.isfinite(dx[[3, 5]]).any()
    assert torch.isnan(dwg[0]).all() and torch.equal(dwg[8:], clean[1][8:])
    zero = fwt.gated_backward(make(40, 130, 4, 0.0), x, wg, wu)
    assert all((t == 0).all() for t in zero)


def test_a_workspace_of_the_type():
    x, wg, wu, grad = inputs(1e4, 40, 256, 130)
    want = fwt.gated_backward(grad, x, wg, wu)
    size = fwt.fwt_gated_backward_workspace_bytes(40, 130, torch.float16)
    assert size > fwt.fwt_gated_backward_workspace_bytes(40, 130)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    got = fwt.gated_backward(grad, x, wg, wu, workspace=work)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one that holds the two matrices alone, as bfloat16 needs it: another is taken instead
    small = torch.empty(fwt.fwt_gated_backward_workspace_bytes(40, 130), dtype=torch.uint8, device="cuda")
    got = fwt.gated_backward(grad, x, wg, wu, workspace=small)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(fwt.FwtError):
        fwt.gated_backward(grad, x, wg, wu, workspace=small[:-16])
