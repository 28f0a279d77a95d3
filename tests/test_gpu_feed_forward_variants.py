"""Every kernel that a feed-forward call can take, against 64 bits, with the plan log to say that it
was taken; and the promise that gradients of up to 8 lines are rounded once."""
import json
import os
import re
import subprocess
import sys

import pytest
import torch

import feed_forward_cuts as cuts
import feed_forward_plain as plain
import test_gpu_feed_forward as base
import walsh_hadamard_transform_gb300 as fwt
from feed_forward_plain import HALF_ULP, TINY
from test_gpu_feed_forward import U, gated_inputs, gated_slack

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

# A process of its own, as the log is asked for once: the test of each case, its lines after it.
CHILD = """
import json, sys
sys.path[:0] = [%r, %r]
import test_gpu_feed_forward as t
for case in json.loads(sys.argv[2]):
    print("case", json.dumps(case), file=sys.stderr, flush=True)
    getattr(t, sys.argv[1])(*case)
""" % (HERE, os.path.dirname(HERE))


def taken(line):
    """The kernel of a line of the log, as feed_forward_cuts names it."""
    name, how = line.split(" | ")
    head = re.match(r"fwt: (matmul_blocks|gated(?: gradients| dx| dw)?(?: f16| bf16)|gated bounds)", name)[1]
    if head == "matmul_blocks":
        head = re.search(r"scale_lines=\d+", name)[0]
    return f"{head} {how}"


@pytest.mark.parametrize("test,choose,kernels", [
    ("test_matmul_blocks", cuts.matmul_cases, cuts.matmul_kernels),
    ("test_gated", cuts.gated_cases, cuts.gated_kernels),
    ("test_gated_backward", cuts.backward_cases, cuts.backward_kernels)])
def test_every_kernel(test, choose, kernels):
    found, left = choose(torch.cuda.get_device_properties(0).multi_processor_count)
    assert not left, left
    run = subprocess.run([sys.executable, "-c", CHILD, test, json.dumps([c for c, _ in found])],
                         env=dict(os.environ, FWT_LOG="1"), capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-3000:]
    seen, parts = set(), run.stderr.split("case ")[1:]
    assert len(parts) == len(found)
    for (case, expected), part in zip(found, parts):
        took = {taken(line) for line in part.splitlines() if line.startswith("fwt: ") and " | " in line}
        assert expected <= took, (case, expected, took)
        seen |= took
    assert kernels() <= seen


@pytest.mark.parametrize("rows,cols,dtype,rotate,axis,lines", [
    (130, 200, "f16", 6, 0, 128), (257, 300, "f16", 7, 0, 128), (200, 333, "f32", 7, 1, 128),
    (140, 260, "f32", 5, 0, 128)])
@pytest.mark.parametrize("aligned", [True, False])
def test_quantize_blocks_of_the_remaining_kinds(rows, cols, dtype, rotate, axis, lines, aligned):
    base.test_quantize_blocks(rows, cols, dtype, rotate, axis, lines, aligned)


@pytest.mark.parametrize("m", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("d,f,dtype,act", [(300, 900, "bf16", "silu"), (1001, 264, "f16", "gelu"),
                                           (64, 2057, "bf16", "relu"), (520, 130, "f16", "silu")])
def test_gradients_of_few_lines_are_rounded_once(m, d, f, dtype, act):
    """dg and du stay in fp32: their own errors are the products' and 8 U for what is multiplied
    and the activation's steps, and no half unit of a 16-bit type."""
    x, wg, wu, grad = gated_inputs(m, d, f, dtype)
    got = fwt.gated_backward(grad, x, wg, wu, activation=act)
    dg, du = plain.gated_parts(grad, x, wg, wu, act)
    _, eu, ev, es = gated_slack(x, wg, wu, act)
    dh, xd, wgd, wud = (t.double().cpu().abs() for t in (grad, x, wg, wu))
    slope = plain.activation(x.double().cpu() @ wg.double().cpu().t(), act)[1].abs()
    u = (x.double().cpu() @ wu.double().cpu().t()).abs()
    edg = dh * (u * es + (slope + es) * eu) + 8 * U * dg.abs()
    edu = dh * ev + 8 * U * du.abs()
    want = plain.gated_backward(grad, x, wg, wu, act)
    sums = (edg @ wgd + edu @ wud + 4 * f * U * (dg.abs() @ wgd + du.abs() @ wud),
            edg.t() @ xd + 2 * m * U * (dg.abs().t() @ xd),
            edu.t() @ xd + 2 * m * U * (du.abs().t() @ xd))
    for name, a, w, s in zip(("dx", "dw_gate", "dw_up"), got, want, sums):
        bound = 1.01 * s + HALF_ULP[dtype] * w.abs() + TINY[dtype]
        err = (a.double().cpu() - w).abs()
        assert (err <= bound).all(), (name, (err / bound.clamp(min=1e-300)).max())
