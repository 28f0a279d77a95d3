"""Valid cache calls where no CUDA device is to be had end in a status (CPU only; a process of its own
that sees no device, so nothing can be launched on the made-up addresses)."""
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
import test_cache_arguments as t
name, defaults = t.ENTRY[sys.argv[1]]
print(t.call(getattr(t.fwt.library(), name), defaults, **eval(sys.argv[2])))
""" % (HERE, os.path.dirname(HERE))


@pytest.mark.parametrize("which,changed", [("append", {}), ("read", {}), ("attend", {}), ("attend", dict(longest=20)),
                                           ("attend", dict(q_heads=2, longest=1))])
def test_no_device_is_an_error(which, changed):
    fbuild.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    run = subprocess.run([sys.executable, "-c", CHILD, which, repr(changed)], env=env, capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stderr[-500:])
    assert run.stdout.split() == [str(fwt.FWT_ERR_CUDA)]
