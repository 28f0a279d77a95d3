"""quantize_blocks of values next to the least scale."""
import pytest
import torch

import feed_forward_plain as plain
import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import check_quantized, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rotate", [0, 1, 7])
@pytest.mark.parametrize("axis,lines", [(1, 1), (1, 128), (0, 1), (0, 128)])
def test_values_next_to_the_least_scale(axis, lines, rotate, dtype):
    """Blocks whose values lie between 2^-134 (for bfloat16 its least, 2^-133) and 2^-110: the
    least scale, 2^-126, holds them to 2^-136."""
    rows, cols = (256, 384) if axis else (384, 256)
    x = torch.randn(rows, cols, generator=gen(1), dtype=torch.float64)
    across = torch.arange(rows if axis else cols)
    size = 2.0 ** -(110 + across % 25).double()
    x = (x.sign() * x.abs().clamp(min=0.5)) * (size[:, None] if axis else size)
    if lines == 128:  # a tile whose lines are all small, and one that has large lines too
        x[:128 if axis else rows, :cols if axis else 128] *= 2.0 ** -16
    x = x.to(plain.REALS[dtype])
    q, s = fwt.quantize_blocks(x.cuda(), rotate=rotate, axis=axis, lines=lines)
    check_quantized(x, q, s, rotate, axis, lines)


def test_one_value_below_the_least_piece():
    x = torch.zeros(2, 128)
    x[0, 0], x[0, 1], x[1, 5] = 2.0 ** -134, 1.875 * 2.0 ** -133, -(2.0 ** -135)
    q, s = fwt.quantize_blocks(x.cuda(), rotate=0)
    v = plain.values(q)
    assert (s == 2.0 ** -126).all()
    # (below 2^-6 the codes lie 2^-9 apart: 1.875 * 2^-7 is 7.5 of these, and goes to the even 8)
    assert v[0, 0] == 2.0 ** -8 and v[0, 1] == 8 * 2.0 ** -9 and v[1, 5] == -(2.0 ** -9)
