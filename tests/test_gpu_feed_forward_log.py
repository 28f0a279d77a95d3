"""The plan log and the event tracing cover the feed-forward operators."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = """
import torch, walsh_hadamard_transform_gb300 as fwt
x, w = torch.randn(40, 256, device="cuda").half(), torch.randn(384, 256, device="cuda").half()
h = fwt.gated(x, w, w)
q, s = fwt.quantize_blocks(h, rotate=5)
fwt.matmul_blocks(q, s, q, s)
fwt.matmul_blocks(q[:3], s[:3], q, s)
fwt.gated_backward(h, x, w, w)
fwt.gated_backward(h[:2], x[:2], w, w, want=("x",))
torch.cuda.synchronize()
"""


def test_plan_log_has_a_line_for_each_kernel():
    for value in ("1", "0"):
        r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env=dict(os.environ, FWT_LOG=value),
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        lines = [ln[5:] for ln in r.stderr.splitlines() if ln.startswith("fwt: ")]
        if value == "0":
            assert lines == []
            continue
        starts = ["gated f16 rows=40 cols=384 stages=4 | tiles ", "quantize_blocks lines=40 length=384 rotate=5 axis=1 ",
                  "matmul_blocks m=40 n=40 k=384 scale_lines=1 | tiles ",
                  "matmul_blocks m=3 n=40 k=384 scale_lines=1 | tokens=8 ", "gated bounds f16 m=40 f=384 d=256",
                  "gated gradients f16 rows=40 ", "gated dx f16 rows=40 cols=256 stages=12 ",
                  "gated dw f16 rows=384 cols=256 stages=1 ", "gated gradients f16 m=2 f=384 d=256 | tokens=8",
                  "gated dx f16 m=2 f=384 d=256 | tokens=2"]
        assert len(lines) == len(starts), lines
        assert all(line.startswith(start) for line, start in zip(lines, starts)), lines


def test_events_around_each_kernel():
    lib = fwt.library()
    x, w = torch.randn(40, 256, device="cuda").half(), torch.randn(384, 256, device="cuda").half()
    h = fwt.gated(x, w, w)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(12)]
    for e in events:
        e.record()
    torch.cuda.synchronize()
    handles = (ctypes.c_void_p * 12)(*(e.cuda_event for e in events))
    assert lib.fwt_trace_events(handles, 12) == fwt.FWT_OK
    try:
        fwt.gated(x, w, w)
        fwt.gated_backward(h, x, w, w)  # bounds, gradients, dx, dw
        assert lib.fwt_trace_count() == 10
        fwt.quantize_blocks(h)
        fwt.quantize_blocks(h)  # no events are left
        assert lib.fwt_trace_count() == 12
    finally:
        lib.fwt_trace_events(None, 0)
    torch.cuda.synchronize()
    times = [a.elapsed_time(b) for a, b in zip(events[::2], events[1::2])]
    assert all(0 < t < 1000 for t in times), times
