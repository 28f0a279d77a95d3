"""Operands whose rows do not start on 16-byte boundaries: refused, by name."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt

pytestmark = pytest.mark.gpu


def empty(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def refused(match):
    return pytest.raises(fwt.FwtError, match=match)


def test_the_operand_is_named():
    x, odd = empty(5, 40), empty(5, 39)
    w, w_odd = empty(20, 40), empty(20, 39)
    with refused("x starts at 0 bytes .* rows are 78 bytes apart; .* multiple of 8 elements") as error:
        fwt.gated(odd, w_odd, w_odd)
    assert error.value.status == fwt.FWT_ERR_MISALIGNED
    with refused("w_up starts at 2 bytes past a multiple of 16 and its rows are 96 bytes"):
        fwt.gated(x, w, empty(20, 48)[:, 1:41])
    with refused("grad starts at 0 bytes .* rows are 42 bytes apart"):
        fwt.gated_backward(empty(5, 21), x, empty(21, 40), empty(21, 40))
    q = empty(5, 200, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = empty(5, 2, dtype=torch.float32)
    with refused("b starts at 8 bytes .* multiple of 16 elements"):
        fwt.matmul_blocks(empty(5, 208, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :192], s,
                          empty(5, 208, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, 8:200], s)
    with refused("a starts at 0 bytes .* rows are 200 bytes"):
        fwt.matmul_blocks(q, s, q, s)
    with refused("codes starts at 0 bytes .* rows are 40 bytes"):
        fwt.quantize_blocks(x, out=(empty(5, 40, dtype=torch.uint8).view(torch.float8_e4m3fn),
                                    empty(5, 1, dtype=torch.float32)))
    with refused("invalid argument"):  # other errors are told as they were
        fwt.gated(x, w, w, out=w[:5, :20])


def test_one_row_has_no_distance():
    x, w = empty(1, 39), empty(20, 40)[:, :39]
    assert fwt.gated(x, w, w).shape == (1, 20)
