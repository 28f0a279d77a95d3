"""Shared arrays of the kernels that are written or read 16 bytes at a time say so (CPU only)."""
import os
import re

import pytest

from test_feed_forward_sources import SOURCES, code


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_vectors_lie_in_arrays_of_their_alignment(path):
    """Where nothing says so, an array's alignment is its elements', and which offset it lands on is
    the compiler's affair."""
    text = code(path)
    for match in re.finditer(r"__shared__\s+(__align__\(\d+\)\s+)?(?:volatile\s+)?(\w+)\s+(\w+)\[", text):
        aligned, _, name = match.groups()
        kernel = text[match.end():].split("__global__")[0]  # names come again in other kernels
        wide = re.search(r"\((?:const )?(?:float4|uint4|float2|uint2)\*\)\s*&?" + name + r"\b", kernel)
        assert aligned or not wide, name
