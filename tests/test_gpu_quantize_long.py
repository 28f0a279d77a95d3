"""quantize_blocks on axes and lines whose bytes pass 31 bits."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import check_quantized, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axis", [1, 0])
def test_an_axis_of_more_than_2_to_the_30(axis):
    """Few lines, or few rows of many columns: the last partial strip of an extent whose bytes pass
    31 bits."""
    n = (1 << 30) + 264
    x = torch.zeros((3, n) if axis else (5, n), dtype=torch.bfloat16, device="cuda")
    at = torch.cat([torch.arange(0, 512), torch.arange(n - 512, n), torch.arange((n // 2) & ~127, (n // 2 & ~127) + 256)])
    x[:, at.cuda()] = torch.randn(x.shape[0], at.numel(), generator=gen(3)).bfloat16().cuda()
    q, s = fwt.quantize_blocks(x, rotate=7 if axis else 0, axis=axis)
    for start in (0, n // 2 & ~127, (n - 512) & ~127):
        end = min(start + 512, n)
        part = x[:, start:end].contiguous()
        qp, sp = fwt.quantize_blocks(part, rotate=7 if axis else 0, axis=axis)
        if axis:
            assert torch.equal(q.view(torch.uint8)[:, start:start + qp.shape[1]], qp.view(torch.uint8))
            assert torch.equal(s[:, start // 128:start // 128 + sp.shape[1]], sp)
        else:
            assert torch.equal(q.view(torch.uint8)[start:end], qp.view(torch.uint8))
            assert torch.equal(s[start:end], sp)
        check_quantized(part, qp, sp, 7 if axis else 0, axis, 1)
