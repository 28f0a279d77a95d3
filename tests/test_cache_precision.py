"""The bound on attention's errors tells one float16 from two (64-bit emulation on the CPU)."""
import pytest
import torch

from cache_precision import FEW, MANY, MOST, SIZES, attend, cut, problem, ratio


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("shape", FEW + MANY)
def test_the_bound_tells_one_float16_from_two(shape, size):
    pr, q = problem(shape, size, "f16", "cpu")
    rotate = 6 if pr.dim == 64 else 7
    exact = attend(pr, q, rotate)[0].half()
    both = attend(pr, q, rotate, cut, cut)[0].half()
    only_p = attend(pr, q, rotate, of_p=cut)[0].half()
    assert ratio(exact, pr, q, rotate, "f16", 0, 0) <= MOST
    assert ratio(only_p, pr, q, rotate, "f16", 0, 1) <= MOST
    assert ratio(both, pr, q, rotate, "f16", 1, 1) <= MOST
    # one rounding too many
    if size == SIZES[0]:
        assert ratio(only_p, pr, q, rotate, "f16", 0, 0) > MOST
    else:
        assert ratio(both, pr, q, rotate, "f16", 0, 1) > MOST


def test_cut_rounds_to_eleven_bits():
    x = torch.randn(1000, dtype=torch.float64)
    assert torch.equal(cut(x), x.half().double())
