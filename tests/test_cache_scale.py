"""Scales of the scores that are finite, but not in powers of two (CPU only)."""
import pytest

import walsh_hadamard_transform_gb300 as fwt
from test_cache_arguments import ATTEND, E, call, lib  # noqa: F401


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scales_that_overflow_are_refused(lib, scale):  # noqa: F811
    assert call(lib.fwt_cache_attention, ATTEND, scale=scale) == E


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 1e-45, 0.0])
def test_others_are_taken(lib, scale):  # noqa: F811
    # (refused after the scale, for its alignment)
    assert call(lib.fwt_cache_attention, ATTEND, scale=scale, places=dict(starts=1)) == fwt.FWT_ERR_MISALIGNED
