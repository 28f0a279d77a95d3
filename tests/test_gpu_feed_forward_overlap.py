"""Kernels that start while the previous one on their stream still writes what they read: chains
over the same buffers with other data each time, against the same calls one after the other."""
import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from test_gpu_feed_forward import gen

pytestmark = pytest.mark.gpu
TURNS = 40


def normal(rows, cols, seed, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(rows, cols, generator=gen(seed)) * scale).to(dtype).cuda()


def chain(m, d, f, dtype, turns):
    """y, dx and dw of every turn: h, its codes and scales, a weight's codes and scales, dh and the
    workspace of the gradients are the same memory in all of them."""
    wg, wu = normal(f, d, 1, d ** -0.5, dtype), normal(f, d, 2, d ** -0.5, dtype)
    xs = [normal(m, d, 10 + i, 1 + i % 3, dtype) for i in range(4)]
    downs = [normal(d, f, 20 + i, f ** -0.5) for i in range(3)]
    empty = lambda *s, t=dtype: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    h, q, s = empty(m, f), empty(m, f, t=e4m3), empty(m, -(-f // 128), t=f32)
    wq, ws = empty(d, f, t=e4m3), empty(-(-d // 128), -(-f // 128), t=f32)
    tq, ts = empty(f, d, t=e4m3), empty(-(-f // 128), -(-d // 128), t=f32)
    yq, ys = empty(m, d, t=e4m3), empty(m, -(-d // 128), t=f32)
    dh = empty(m, f)
    work = empty(fwt.fwt_gated_backward_workspace_bytes(m, f, dtype), t=torch.uint8)
    y = [empty(m, d) for _ in range(turns)]
    grads = [(empty(m, d), empty(f, d), empty(f, d)) for _ in range(turns)]
    torch.cuda.synchronize()
    for i in range(turns):
        x, down = xs[i % 4], downs[i % 3]
        fwt.quantize_blocks(down, rotate=7, lines=128, out=(wq, ws))
        fwt.gated(x, wg, wu, out=h)
        fwt.quantize_blocks(h, rotate=7, out=(q, s))
        fwt.matmul_blocks(q, s, wq, ws, out=y[i])
        fwt.quantize_blocks(down, rotate=7, axis=0, lines=128, out=(tq, ts))
        fwt.quantize_blocks(y[i], rotate=7, out=(yq, ys))
        fwt.matmul_blocks(yq, ys, tq, ts, out=dh)
        fwt.gated_backward(dh, x, wg, wu, out=grads[i], workspace=work)
    torch.cuda.synchronize()
    return [t for i in range(turns) for t in (y[i], *grads[i])]


@pytest.mark.parametrize("m,d,f,dtype", [
    (1, 256, 640, torch.bfloat16), (8, 512, 1024, torch.float16), (24, 256, 512, torch.bfloat16),
    (200, 384, 640, torch.float16), (1200, 256, 1024, torch.bfloat16)])
def test_chains_over_the_same_buffers(m, d, f, dtype):
    assert fwt.pdl() == 1
    fwt.set_pdl(0)
    try:
        want = chain(m, d, f, dtype, 12)  # the data come round after twelve turns
    finally:
        fwt.set_pdl(1)
    got = chain(m, d, f, dtype, TURNS)
    for i, t in enumerate(got):
        assert torch.equal(t, want[i % len(want)]), (i // 4, i % 4)
    assert fwt.device_status() == fwt.FWT_OK
