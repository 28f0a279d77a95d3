"""Attention's errors over a call are no more than the documented roundings leave, for each kernel and type."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from cache_precision import FEW, MANY, MOST, SIZES, problem, ratio

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("shape", FEW + MANY)
def test_roundings(shape, size, dtype):
    pr, q = problem(shape, size, dtype, "cuda")
    few, fine = shape in FEW, dtype == "f16"
    got = fwt.cache_attention(q, *pr.places(), longest=0 if few else 90)
    with_q, with_p = not (fine and (few or pr.dim == 64)), not (fine and few)
    assert ratio(got, pr, q, 6 if pr.dim == 64 else 7, dtype, with_q, with_p) <= MOST
