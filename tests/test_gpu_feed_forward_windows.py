"""Outputs in the gaps between the rows of other operands."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 3])
def test_a_row_beside_the_rows_of_a_weight(m):
    """A window of one row has no second row: whatever distance it would have, it lies in the gap
    and overlaps nothing."""
    make = lambda rows, cols, s: torch.randn(rows, cols, generator=gen(s)).bfloat16().cuda()  # noqa: E731
    x, wu, wide = make(m, 64, 1), make(40, 64, 2) / 8, make(40, 128, 3) / 8
    wg = wide[:, :64]
    want = fwt.gated(x, wg, wu)
    out = wide[7:7 + m, 64:104]
    assert fwt.gated(x, wg, wu, out=out) is out
    assert torch.equal(out, want)
    with pytest.raises(fwt.FwtError):
        fwt.gated(x, wg, wu, out=wide[7:7 + m, 60:100])
    with pytest.raises(fwt.FwtError):
        fwt.gated(x, wg, wu, out=wide[7:7 + m, 100:].as_strided((m, 40), (128, 1)))
