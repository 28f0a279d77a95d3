"""Feed-forward operators on CUDA tensors: the rotation fused with 8-bit block
quantisation, the product of such operands, and the gated projections with their
gradients.

    h = gated(x, w_gate, w_up)                       act(x w_gate^T) * (x w_up^T)
    q, s = quantize_blocks(h, rotate=7)              rotated, 8 bits, a scale for each 128
    y = matmul_blocks(q, s, w_q, w_s)                w_q, w_s = quantize_blocks(w, rotate=7, lines=128)

The rotation is its own inverse, so rotating both operands of a product along the
contraction leaves the product as it is.  Matrices are 2-D tensors whose rows are
contiguous (stride 1 along the columns) and may be a window of a larger matrix;
operands of products start every row on a 16-byte boundary.  Outputs made here have
such rows too (padded where the width asks for it).  Every call runs on ``stream``
(default: the current PyTorch stream) and does not synchronise; what it allocates belongs
to that stream, as under ``torch.cuda.stream``.  A kernel whose waits give up leaves its output
unwritten: ``device_status()``, which synchronises, tells.
"""
from __future__ import annotations

import walsh_hadamard_transform_gb300 as _fwt

_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}
_torch = _REALS = _E4M3 = _F32 = _lib = _device = _raw_stream = None


def _load():
    """torch and the C library, on first use."""
    global _torch, _REALS, _E4M3, _F32, _lib, _device, _raw_stream
    torch = _fwt._torch_mod()
    _E4M3, _F32 = torch.float8_e4m3fn, torch.float32
    _REALS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    _torch = torch
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _lib = _fwt.library()


def _matrix(t, name, device, dtype=None, shape=None):
    """Row stride of a 2-D tensor with contiguous rows on CUDA device number ``device``."""
    size = t.shape
    if size != shape:
        if len(size) != 2:
            raise ValueError(f"{name}: expected a matrix, got {len(size)} dimensions")
        if shape is not None:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(size)}")
    if device < 0 or t.get_device() != device:
        raise ValueError(f"{name}: every tensor must be on one CUDA device")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    row, col = t.stride()
    rows, cols = size
    if col != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows <= 1:  # no second row: any stride will do
        return cols + -cols % 16
    return row


def _empty(rows, cols, dtype, device, multiple, stream):
    """A new rows x cols tensor for work on ``stream``, its rows a multiple of ``multiple``
    elements apart, and that distance."""
    if stream is not None:
        with _allocations(device, stream):
            return _empty(rows, cols, dtype, device, multiple, None)
    over = cols % multiple
    if over:
        ld = cols + multiple - over
        return _torch.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=device), ld
    return _torch.empty((rows, cols), dtype=dtype, device=device), cols


def _allocations(device, stream):
    """A context in which new tensors belong to ``stream``, a PyTorch stream or a raw handle:
    memory of the current stream may still be in use there, and may be handed out again there
    before ``stream`` is done with it."""
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)  # (0 and 1 are names of the default stream)
        stream = (_torch.cuda.ExternalStream(handle, device=device) if handle > 1
                  else _torch.cuda.default_stream(device))
    return _torch.cuda.stream(stream)


def _run(device, stream, entry, *args):
    """Calls the C entry on ``stream`` (default: the current one) with the device current."""
    if stream is not None:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    else:
        handle = _raw_stream(device)
    if device == _device():
        return entry(*args, handle)
    with _torch.cuda.device(device):
        return entry(*args, handle)


def _error(status, what, aligned, elements=()):
    """The error of a call.  Where a matrix does not start its rows as the call asks for, says
    which one: ``aligned`` are those on 16-byte boundaries, ``elements`` those on their elements'."""
    if status == _fwt.FWT_ERR_MISALIGNED:
        for tensors, unit in ((aligned, 16), (elements, 0)):
            for name, t in tensors:
                size = t.element_size()
                row = t.stride(0) * size if t.dim() == 2 and t.shape[0] > 1 else 0
                if t.data_ptr() % (unit or size) or (unit and row % unit):
                    what += (f": {name} starts at {t.data_ptr() % (unit or size)} bytes past a multiple "
                             f"of {unit or size}" + (f" and its rows are {row} bytes apart" if row else "")
                             + (f"; as a window of rows padded to a multiple of {unit // size} elements "
                                "it would be taken" if unit else ""))
                    return _fwt.FwtError(status, what)
    return _fwt.FwtError(status, what)


def quantize_blocks(x, rotate: int = 0, axis: int = 1, lines: int = 1, out=None, stream=None):
    """Rotates ``x`` (rows, cols) along ``axis`` and quantises it to 8-bit e4m3.

    Each aligned group of ``2**rotate`` elements (0 <= rotate <= 7) along the axis is
    multiplied by the normalised H, the length extended with zeros to whole groups; then
    each block of 128 elements along the axis by ``lines`` (1 or 128) lines across it gets
    an fp32 scale max|y| / 448 and codes e4m3(y / scale).  ``axis=1``: along the columns,
    codes (rows, L).  ``axis=0``: down the rows, codes transposed (cols, L), so that they
    run along the contraction of a gradient product.

    ``x``: float32, bfloat16 or float16.  ``out``: (codes, scale) to write to.  Returns
    (codes, scale): float8_e4m3fn (lines of codes, L) and float32 of a row for each
    ``lines`` lines and a column for each block.
    """
    if _lib is None:
        _load()
    kind, device = _REALS.get(x.dtype), x.get_device()
    if kind is None:
        raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16 or float16")
    if axis not in (0, 1) or lines not in (1, 128) or not 0 <= rotate <= 7:
        raise ValueError("axis is 0 or 1, lines 1 or 128 and rotate 0 .. 7")
    ld = _matrix(x, "x", device)
    rows, cols = x.shape
    across, length = (rows, cols) if axis else (cols, rows)
    length += -length % (1 << rotate)
    shape = (-(-across // lines), -(-length // 128))
    if out is None:
        q, ld_q = _empty(across, length, _E4M3, x.device, 16, stream)
        scale, ld_s = _empty(*shape, _F32, x.device, 4, stream)
    else:
        q, scale = out
        ld_q = _matrix(q, "codes", device, _E4M3, (across, length))
        ld_s = _matrix(scale, "scale", device, _F32, shape)
    st = _run(device, stream, _lib.fwt_quantize_blocks, x.data_ptr(), kind, rows, cols, ld, rotate,
              axis, lines, q.data_ptr(), ld_q, scale.data_ptr(), ld_s)
    if st != _fwt.FWT_OK:
        raise _error(st, f"fwt_quantize_blocks({rows} x {cols}, axis={axis})", [("codes", q)],
                     [("x", x), ("scale", scale)])
    return q, scale


def matmul_blocks(a, a_scale, b, b_scale, out_dtype=None, out=None, stream=None):
    """C = A B^T of 8-bit operands with block scales, as ``quantize_blocks`` writes them.

    ``a``: float8_e4m3fn (m, k), ``a_scale``: float32 (m, ceil(k / 128)).  ``b``: (n, k),
    ``b_scale`` a row for each line, (n, ceil(k / 128)), or for each 128 of them.  C is
    (m, n) of ``out_dtype`` (bfloat16 by default, float16 or float32), or ``out``.
    """
    if _lib is None:
        _load()
    device = a.get_device()
    ld_a = _matrix(a, "a", device, _E4M3)
    ld_b = _matrix(b, "b", device, _E4M3)
    m, k = a.shape
    n, k_b = b.shape
    if k_b != k:
        raise ValueError(f"a and b have {k} and {k_b} elements along the contraction")
    blocks = -(-k // 128)
    ld_as = _matrix(a_scale, "a_scale", device, _F32, (m, blocks))
    lines = 1 if b_scale.shape[:1] == (n,) else 128
    ld_bs = _matrix(b_scale, "b_scale", device, _F32, (-(-n // lines), blocks))
    if out is None:
        out_dtype = out_dtype or _torch.bfloat16
        kind = _REALS.get(out_dtype)
        if kind is None:
            raise TypeError(f"unsupported dtype {out_dtype}: use float32, bfloat16 or float16")
        out, ld_c = _empty(m, n, out_dtype, a.device, 4 if kind == 0 else 8, stream)
    else:
        kind = _REALS.get(out.dtype)
        if kind is None or (out_dtype is not None and out.dtype != out_dtype):
            raise TypeError(f"out: unsupported dtype {out.dtype}")
        ld_c = _matrix(out, "out", device, None, (m, n))
    st = _run(device, stream, _lib.fwt_matmul_blocks, a.data_ptr(), ld_a, a_scale.data_ptr(), ld_as,
              b.data_ptr(), ld_b, b_scale.data_ptr(), ld_bs, lines, out.data_ptr(), kind, ld_c, m, n,
              k)
    if st != _fwt.FWT_OK:
        raise _error(st, f"fwt_matmul_blocks(m={m}, n={n}, k={k})", [("a", a), ("b", b)],
                     [("a_scale", a_scale), ("b_scale", b_scale), ("out", out)])
    return out


def _gated_arguments(x, w_gate, w_up, activation):
    if _lib is None:
        _load()
    dtype, device = x.dtype, x.get_device()
    kind = _REALS.get(dtype)
    if kind != 1 and kind != 2:
        raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float16")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r}: use one of {sorted(_ACTIVATIONS)}")
    ld_x = _matrix(x, "x", device)
    m, d = x.shape
    shape = (w_gate.shape[0], d)
    ld_g = _matrix(w_gate, "w_gate", device, dtype, shape)
    ld_u = _matrix(w_up, "w_up", device, dtype, shape)
    return dtype, kind, act, device, m, shape[0], d, ld_x, ld_g, ld_u


def gated(x, w_gate, w_up, activation: str = "silu", out=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T): both products, the activation and their product
    in one kernel, fp32 inside and rounded once.

    ``x`` (m, d), ``w_gate`` and ``w_up`` (f, d): bfloat16 or float16, all of one type.
    ``activation``: "silu", "gelu" (the tanh form) or "relu".  Returns h (m, f)."""
    dtype, kind, act, device, m, f, d, ld_x, ld_g, ld_u = _gated_arguments(x, w_gate, w_up,
                                                                           activation)
    if out is None:
        out, ld_h = _empty(m, f, dtype, x.device, 8, stream)
    else:
        ld_h = _matrix(out, "out", device, dtype, (m, f))
    st = _run(device, stream, _lib.fwt_gated, x.data_ptr(), ld_x, w_gate.data_ptr(), ld_g,
              w_up.data_ptr(), ld_u, out.data_ptr(), ld_h, kind, act, m, f, d)
    if st != _fwt.FWT_OK:
        raise _error(st, f"fwt_gated(m={m}, f={f}, d={d})",
                     [("x", x), ("w_gate", w_gate), ("w_up", w_up)], [("out", out)])
    return out


def gated_backward(grad, x, w_gate, w_up, activation: str = "silu", out=None, workspace=None,
                   want=("x", "w"), stream=None):
    """Gradients of ``gated`` for ``grad``, the gradient of h (m, f).

    Returns (dx, dw_gate, dw_up), of the inputs' shapes and type; those not named in
    ``want`` ("x", and "w" for both weights) are not computed and None.  ``out``: the
    three tensors to write to.  ``workspace``: a CUDA tensor of at least
    ``fwt_gated_backward_workspace_bytes(m, f, dtype)`` bytes for the gradients of the two
    products (allocated here when None, or when a float16 call is given one of the size for
    bfloat16)."""
    dtype, kind, act, device, m, f, d, ld_x, ld_g, ld_u = _gated_arguments(x, w_gate, w_up,
                                                                           activation)
    ld_dy = _matrix(grad, "grad", device, dtype, (m, f))
    want_x, want_w = "x" in want, "w" in want
    dx = dw_gate = dw_up = None
    p_dx = p_dg = p_du = None
    ld_dx = ld_dg = ld_du = 0
    if out is not None:
        dx, dw_gate, dw_up = out
        if (want_x != (dx is not None) or want_w != (dw_gate is not None)
                or want_w != (dw_up is not None)):
            raise ValueError("out must hold the gradients named in want, and no other")
    if want_x:
        if dx is None:
            dx, ld_dx = _empty(m, d, dtype, x.device, 8, stream)
        else:
            ld_dx = _matrix(dx, "dx", device, dtype, (m, d))
        p_dx = dx.data_ptr()
    if want_w:
        if dw_gate is None:
            dw_gate, ld_dg = _empty(f, d, dtype, x.device, 8, stream)
            dw_up, ld_du = _empty(f, d, dtype, x.device, 8, stream)
        else:
            ld_dg = _matrix(dw_gate, "dw_gate", device, dtype, (f, d))
            ld_du = _matrix(dw_up, "dw_up", device, dtype, (f, d))
        p_dg, p_du = dw_gate.data_ptr(), dw_up.data_ptr()
    size = _lib.fwt_gated_backward_workspace_bytes_for(kind, m, f)
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        given = workspace.numel() * workspace.element_size()
        if _lib.fwt_gated_backward_workspace_bytes(m, f) <= given < size:
            workspace = None
        else:
            size = given
    if workspace is None:
        workspace, _ = _empty(1, size, _torch.uint8, x.device, 1, stream)
    st = _run(device, stream, _lib.fwt_gated_backward, grad.data_ptr(), ld_dy, x.data_ptr(), ld_x,
              w_gate.data_ptr(), ld_g, w_up.data_ptr(), ld_u, p_dx, ld_dx, p_dg, ld_dg, p_du, ld_du,
              kind, act, m, f, d, workspace.data_ptr(), size)
    if st != _fwt.FWT_OK:
        raise _error(st, f"fwt_gated_backward(m={m}, f={f}, d={d})",
                     [("grad", grad), ("x", x), ("w_gate", w_gate), ("w_up", w_up),
                      ("workspace", workspace)])
    return dx, dw_gate, dw_up


def fwt_gated_backward_workspace_bytes(m: int, f: int, dtype=None) -> int:
    """Bytes of the workspace of ``gated_backward`` for x of (m, d) and weights of (f, d) of
    ``dtype``, bfloat16 (also None) or float16."""
    lib = _fwt.library()
    if dtype is None:
        return int(lib.fwt_gated_backward_workspace_bytes(int(m), int(f)))
    if _lib is None:
        _load()
    kind = _REALS.get(dtype)
    if kind != 1 and kind != 2:
        raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float16")
    return int(lib.fwt_gated_backward_workspace_bytes_for(kind, int(m), int(f)))
