"""A contraction whose products take longer than a wait may last without progress."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt

pytestmark = pytest.mark.gpu


def test_a_tile_of_more_than_a_second():
    """The fewest lines that tiles are used for, by as many stages as take over a second: 2^31 - 1024
    elements, some 0.2 us for 64 of them shared out over four CTAs.  Almost all are zero; ones at both
    ends and in every quarter add up to numbers that 16 bits hold."""
    d, m = (1 << 31) - 1024, 9
    need = (m + 2) * d * 2
    if torch.cuda.mem_get_info()[0] < need * 1.2:
        pytest.skip("needs 48 GB of device memory")
    x = torch.zeros(m, d, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, d, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 63, d // 4 - 1, d // 4, d // 2, 3 * (d // 4) + 5, d - 1], device="cuda")
    x[:, at] = torch.arange(1, m + 1, device="cuda", dtype=torch.bfloat16)[:, None].expand(m, 7)
    w[:, at] = torch.tensor([[1.0], [2.0]], dtype=torch.bfloat16, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    h = torch.empty(m, 1, dtype=torch.bfloat16, device="cuda")
    start.record()
    fwt.gated(x, w[:1], w[1:], activation="relu", out=h)
    end.record()
    assert fwt.device_status() == fwt.FWT_OK
    want = torch.tensor([(7.0 * i) * (14.0 * i) for i in range(1, m + 1)]).bfloat16()
    assert torch.equal(h[:, 0].cpu(), want)
    print(f"{start.elapsed_time(end):.0f} ms")
