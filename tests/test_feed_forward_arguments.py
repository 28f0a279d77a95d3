"""Argument checks of the feed-forward operators, all before any CUDA call (CPU only)."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from walsh_hadamard_transform_gb300 import build as fbuild

A, GiB = 0x100000, 1 << 30  # fake, aligned addresses; validation never dereferences them
OK, E, MIS = fwt.FWT_OK, fwt.FWT_ERR_INVALID_ARG, fwt.FWT_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fwt.library()


def call(entry, defaults, /, **changed):
    args = dict(defaults)
    assert not set(changed) - set(args)
    args.update(changed)
    return entry(*args.values())


QUANTIZE = dict(x=A, x_type=fwt.FWT_BF16, rows=10, cols=200, ld_x=208, rot_bits=7, axis=1, lines=1,
                q=A + GiB, ld_q=256, scale=A + 2 * GiB, ld_scale=2, stream=None)
MATMUL = dict(a=A, ld_a=256, a_scale=A + GiB, ld_as=2, b=A + 2 * GiB, ld_b=256, b_scale=A + 3 * GiB,
              ld_bs=2, b_lines=128, c=A + 4 * GiB, c_type=fwt.FWT_BF16, ld_c=304, m=10, n=300, k=256,
              stream=None)
GATED = dict(x=A, ld_x=64, wg=A + GiB, ld_g=64, wu=A + 2 * GiB, ld_u=64, h=A + 3 * GiB, ld_h=104,
             type=fwt.FWT_BF16, act=fwt.FWT_SILU, m=10, f=100, d=60, stream=None)
BACKWARD = dict(grad=A + 3 * GiB, ld_dy=104, x=A, ld_x=64, wg=A + GiB, ld_g=64, wu=A + 2 * GiB, ld_u=64,
                dx=A + 4 * GiB, ld_dx=64, dwg=A + 5 * GiB, ld_dwg=64, dwu=A + 6 * GiB, ld_dwu=64,
                type=fwt.FWT_BF16, act=fwt.FWT_SILU, m=10, f=100, d=60, ws=A + 7 * GiB, ws_bytes=1 << 20,
                stream=None)

REFUSED = {
    "quantize": [
        (dict(x_type=3), E), (dict(x_type=-1), E), (dict(rot_bits=8), E), (dict(rot_bits=-1), E),
        (dict(axis=2), E), (dict(lines=64), E), (dict(rows=-1), E), (dict(cols=1 << 31), E),
        (dict(ld_x=199), E), (dict(x=None), E), (dict(q=None), E), (dict(scale=None), E),
        (dict(ld_q=192), E), (dict(ld_scale=1), E), (dict(ld_q=257), MIS), (dict(q=A + GiB + 8), MIS),
        (dict(x=A + 1), MIS), (dict(scale=A + 2 * GiB + 2), MIS), (dict(q=A), E), (dict(scale=A + 64), E),
        (dict(ld_x=1 << 59), E), (dict(axis=0, ld_q=16), E),
    ],
    "matmul": [
        (dict(c_type=3), E), (dict(b_lines=2), E), (dict(m=-1), E), (dict(n=1 << 31), E),
        (dict(k=-1), E), (dict(ld_a=255), E), (dict(ld_b=128), E), (dict(ld_c=299), E),
        (dict(ld_as=1), E), (dict(ld_bs=1), E), (dict(a=None), E), (dict(b_scale=None), E),
        (dict(c=None), E), (dict(ld_a=257), MIS), (dict(b=A + 2 * GiB + 4), MIS),
        (dict(c=A + 4 * GiB + 1), MIS), (dict(a_scale=A + GiB + 2), MIS), (dict(c=A), E),
        (dict(c=A + 3 * GiB), E),
    ],
    "gated": [
        (dict(type=fwt.FWT_F32), E), (dict(act=3), E), (dict(act=-1), E), (dict(m=-1), E),
        (dict(ld_x=59), E), (dict(ld_h=99), E), (dict(x=None), E), (dict(wu=None), E), (dict(h=None), E),
        (dict(ld_x=61), MIS), (dict(wg=A + GiB + 8), MIS), (dict(h=A + 3 * GiB + 1), MIS),
        (dict(h=A + 32), E), (dict(h=A + 2 * GiB), E),
    ],
    "backward": [
        (dict(type=fwt.FWT_F32), E), (dict(act=7), E), (dict(dwg=None), E), (dict(dwu=None), E),
        (dict(ws=None), E), (dict(ws_bytes=10 * 104 * 4 - 1), E), (dict(ws=A + 7 * GiB + 8), MIS),
        (dict(grad=A + 3 * GiB + 2), MIS), (dict(ld_dy=102), MIS), (dict(dx=A), E),
        (dict(dwg=A + 6 * GiB), E), (dict(ws=A + GiB), E), (dict(ld_dx=59), E), (dict(dx=A + 4 * GiB + 1), MIS),
        (dict(dx=A + 7 * GiB), E),
    ],
}
ENTRY = {"quantize": ("fwt_quantize_blocks", QUANTIZE), "matmul": ("fwt_matmul_blocks", MATMUL),
         "gated": ("fwt_gated", GATED), "backward": ("fwt_gated_backward", BACKWARD)}


@pytest.mark.parametrize("which", sorted(REFUSED))
def test_refusals_before_any_launch(lib, which):
    name, defaults = ENTRY[which]
    for changed, status in REFUSED[which]:
        assert call(getattr(lib, name), defaults, **changed) == status, (name, changed)


def test_empty_calls_need_no_gpu(lib):
    nothing = dict(x=None, q=None, scale=None)
    assert call(lib.fwt_quantize_blocks, QUANTIZE, rows=0, **nothing) == OK
    assert call(lib.fwt_quantize_blocks, QUANTIZE, cols=0, **nothing) == OK
    assert call(lib.fwt_matmul_blocks, MATMUL, m=0) == OK
    assert call(lib.fwt_matmul_blocks, MATMUL, n=0) == OK
    assert call(lib.fwt_gated, GATED, m=0, x=None, h=None) == OK
    assert call(lib.fwt_gated, GATED, f=0) == OK
    assert call(lib.fwt_gated_backward, BACKWARD, d=0) == OK
    assert call(lib.fwt_gated_backward, BACKWARD, dx=None, dwg=None, dwu=None) == OK


def test_workspace_size(lib):
    size = lib.fwt_gated_backward_workspace_bytes
    assert size(10, 100) == 10 * 104 * 2 * 2 and size(1, 1) == size(8, 8) == 8 * 64
    assert size(0, 5) == 0 and size(5, 0) == 0 and size(-1, 5) == 0 and size(1 << 31, 1) == 0
    assert size(1 << 20, 1 << 14) == 1 << 36


def test_binding_checks():
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="CUDA device"):
        fwt.quantize_blocks(x)
    with pytest.raises(TypeError, match="float64"):
        fwt.quantize_blocks(x.double())
    for bad in (dict(rotate=8), dict(axis=2), dict(lines=2)):
        with pytest.raises(ValueError, match="axis is 0 or 1"):
            fwt.quantize_blocks(x, **bad)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        fwt.gated(x, x, x)
    y = x.bfloat16()
    with pytest.raises(ValueError, match="activation"):
        fwt.gated(y, y, y, activation="tanh")
    with pytest.raises(ValueError, match="CUDA device"):
        fwt.gated(y, y, y)
    with pytest.raises(ValueError, match="CUDA device"):
        fwt.gated_backward(y, y, y, y)
    with pytest.raises(ValueError, match="CUDA device"):
        fwt.matmul_blocks(y, x, y, x)


def test_type_codes_match_the_header():
    import os
    text = open(os.path.join(os.path.dirname(fbuild.PKG), "include", "fwt.h")).read()
    for name in ("FWT_F32", "FWT_BF16", "FWT_F16", "FWT_SILU", "FWT_GELU", "FWT_RELU"):
        assert f"{name} = {getattr(fwt, name)}" in text, name
