"""Valid calls where no CUDA device is to be had end in a status (CPU only; a process of its own that
sees no device, so nothing can be launched on the made-up addresses)."""
import os
import subprocess
import sys

import pytest

import walsh_hadamard_transform_gb300 as fwt
from walsh_hadamard_transform_gb300 import build as fbuild

HERE = os.path.dirname(os.path.abspath(__file__))
CHILD = """
import sys
sys.path[:0] = [%r, %r]
import test_feed_forward_arguments as t
name, defaults = t.ENTRY[sys.argv[1]]
changed = eval(sys.argv[2])
print(t.call(getattr(t.fwt.library(), name), defaults, **changed))
""" % (HERE, os.path.dirname(HERE))
CALLS = [("quantize", {}), ("quantize", dict(axis=0, ld_q=128)),
         ("matmul", {}), ("matmul", dict(m=200)), ("gated", {}), ("gated", dict(m=200)),
         ("backward", {}), ("backward", dict(m=4)), ("backward", dict(type=fwt.FWT_F16)),
         ("matmul", dict(k=0)), ("gated", dict(d=0)), ("backward", dict(m=0))]


@pytest.mark.parametrize("which,changed", CALLS)
def test_no_device_is_an_error(which, changed):
    fbuild.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    run = subprocess.run([sys.executable, "-c", CHILD, which, repr(changed)], env=env,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stderr[-500:])
    assert run.stdout.split() == [str(fwt.FWT_ERR_CUDA)]
