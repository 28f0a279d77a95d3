"""Workspace sizes of gated_backward by type (CPU only)."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from test_feed_forward_arguments import BACKWARD, E, MIS, call, lib  # noqa: F401


def test_sizes(lib):  # noqa: F811
    size = lib.fwt_gated_backward_workspace_bytes_for
    for m, f in ((1, 1), (8, 100), (9, 100), (10, 8), (1 << 20, 1 << 14), (0, 5), (5, 0)):
        base = lib.fwt_gated_backward_workspace_bytes(m, f)
        assert size(fwt.FWT_BF16, m, f) == base
        assert size(fwt.FWT_F16, m, f) == base + (4096 if base and m > 8 else 0)
        assert size(fwt.FWT_F32, m, f) == 0
        assert fwt.fwt_gated_backward_workspace_bytes(m, f) == base
        assert fwt.fwt_gated_backward_workspace_bytes(m, f, torch.float16) == size(fwt.FWT_F16, m, f)
    with pytest.raises(TypeError):
        fwt.fwt_gated_backward_workspace_bytes(9, 9, torch.float32)


def test_float16_asks_for_its_own_size(lib):  # noqa: F811
    f16 = dict(type=fwt.FWT_F16)
    size = lib.fwt_gated_backward_workspace_bytes_for(fwt.FWT_F16, 10, 100)
    assert call(lib.fwt_gated_backward, BACKWARD, ws_bytes=size - 1, **f16) == E
    assert call(lib.fwt_gated_backward, BACKWARD, ws_bytes=size, dx=BACKWARD["ws"] + size - 16, **f16) == E
    assert call(lib.fwt_gated_backward, BACKWARD, ws_bytes=size, ws=BACKWARD["ws"] + 8, **f16) == MIS
