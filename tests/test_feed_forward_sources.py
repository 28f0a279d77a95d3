"""What the sources of the kernels must not hold (CPU only)."""
import glob
import os
import re

import pytest

from walsh_hadamard_transform_gb300 import build as fbuild

SOURCES = sorted(glob.glob(os.path.join(fbuild.CSRC, "*.cu")) + glob.glob(os.path.join(fbuild.CSRC, "*.cuh")))


def code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_reads_through_the_read_only_path(path):
    """Kernels may start while the previous one on their stream still writes what they are to read:
    loads that take their data as unchanging for the kernel's whole life are not for them."""
    text = code(path)
    assert "__ldg" not in text and "ld.global.nc" not in text and "__ldlu" not in text
    assert "__restrict__" not in text  # with const, the compiler's own way to those loads
