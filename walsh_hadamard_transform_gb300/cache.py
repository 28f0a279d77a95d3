"""Keys and values of attention, rotated and held in 8 bits in pages: the operators on CUDA tensors.

    cache = new_cache(pages, page_tokens, heads, dim)
    cache_append(k, v, cache, table, starts, lengths)           rotated, e4m3, a scale a token and head
    out = cache_attention(q, cache, table, starts, lengths)     the new tokens to all of their sequence
    k, v = cache_read(cache, table, starts, lengths, tokens)    the last tokens of each, turned back

Operands are packed: (tokens, heads, dim), the rows of a sequence one after the other, a head's
elements contiguous and on 16-byte boundaries (windows of a fused projection will do).  ``table``
(sequences, most pages), ``starts`` (sequences + 1) and ``lengths`` (sequences) are int32 CUDA
tensors that the host never reads: rows ``starts[b]`` to ``starts[b + 1]`` are the last of the
``lengths[b]`` tokens that sequence b has in the cache, those that the call writes among them, and
row b of ``table`` names its pages.  Rows behind the last sequence are not touched; pages that
are not the cache's (-1, say) hold nothing.  Every call runs on ``stream`` (default: the current
PyTorch stream) and does not synchronise.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import walsh_hadamard_transform_gb300 as _fwt

from . import feed_forward as _ff

_torch = _E4M3 = _E8M0 = _I32 = _lib = None


class Cache(NamedTuple):
    """Codes (pages, heads, page_tokens, dim), float8_e4m3fn, of keys and values, and the scale of
    each token and head (pages, heads, page_tokens), float8_e8m0fnu.  Pages are contiguous; the first
    dimension may have any stride that is a multiple of 16 bytes (a layer of a pool)."""
    k: object
    k_scale: object
    v: object
    v_scale: object


class _CacheArgument(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_void_p) for name in ("k", "v", "k_scale", "v_scale")]
                + [(name, ctypes.c_int64) for name in ("k_stride", "v_stride", "k_scale_stride",
                                                       "v_scale_stride", "pages")]
                + [(name, ctypes.c_int) for name in ("heads", "page_tokens", "dim")])


class _SequencesArgument(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("most_pages", ctypes.c_int64), ("starts", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("sequences", ctypes.c_int64)]


def declare(lib):
    """Argument types of the C entries."""
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    cache, sequences = ctypes.POINTER(_CacheArgument), ctypes.POINTER(_SequencesArgument)
    rows = [vp, i64, i64]
    lib.fwt_cache_append.argtypes = [*rows, *rows, ci, i64, cache, sequences, ci, vp]
    lib.fwt_cache_append.restype = ci
    lib.fwt_cache_read.argtypes = [cache, sequences, ci, *rows, *rows, ci, i64, vp]
    lib.fwt_cache_read.restype = ci
    lib.fwt_cache_attention.argtypes = [*rows, *rows, ci, i64, ci, cache, sequences, ci,
                                        ctypes.c_float, ci, i64, i64, vp, ctypes.c_size_t, vp]
    lib.fwt_cache_attention.restype = ci
    lib.fwt_cache_attention_workspace_bytes.argtypes = [ci, ci, ci, i64]
    lib.fwt_cache_attention_workspace_bytes.restype = ctypes.c_size_t


def _load():
    """torch and the C library, on first use."""
    global _torch, _E4M3, _E8M0, _I32, _lib
    if _ff._lib is None:
        _ff._load()
    torch = _ff._torch
    _E4M3, _E8M0, _I32 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.int32
    _torch = torch
    _lib = _fwt.library()


def new_cache(pages: int, page_tokens: int, heads: int, dim: int, device="cuda") -> Cache:
    """An empty cache, all zeros: ``page_tokens`` a multiple of 16, ``dim`` 64 or 128."""
    if _lib is None:
        _load()
    if dim not in (64, 128) or page_tokens < 16 or page_tokens % 16 or heads < 1 or pages < 0:
        raise ValueError("dim is 64 or 128, page_tokens a multiple of 16, heads at least 1")

    def zeros(dtype, *shape):
        return _torch.zeros(shape, dtype=_torch.uint8, device=device).view(dtype)

    return Cache(*(zeros(_E8M0, pages, heads, page_tokens) if i & 1
                   else zeros(_E4M3, pages, heads, page_tokens, dim) for i in range(4)))


def _cache(cache):
    """The C argument, the device, heads and dim of a cache."""
    k, k_scale, v, v_scale = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("cache: codes are (pages, heads, page_tokens, dim), of keys and values alike")
    pages, heads, page, dim = shape
    of_scales = shape[:3]
    if k_scale.shape != of_scales or v_scale.shape != of_scales:
        raise ValueError("cache: scales are (pages, heads, page_tokens)")
    if dim != 64 and dim != 128 or page < 16 or page % 16:
        raise ValueError("cache: dim is 64 or 128 and page_tokens a multiple of 16")
    if k.dtype is not _E4M3 or v.dtype is not _E4M3 or k_scale.dtype is not _E8M0 or v_scale.dtype is not _E8M0:
        raise TypeError("cache: codes are float8_e4m3fn and scales float8_e8m0fnu")
    device = k.get_device()
    if device < 0 or v.get_device() != device or k_scale.get_device() != device or v_scale.get_device() != device:
        raise ValueError("cache: every tensor must be on one CUDA device")
    of_k, of_v, of_ks, of_vs = k.stride(), v.stride(), k_scale.stride(), v_scale.stride()
    within = (page * dim, dim, 1)
    if of_k[1:] != within or of_v[1:] != within or of_ks[1:] != (page, 1) or of_vs[1:] != (page, 1):
        for t in cache:
            if not _within(t, within if t.dim() == 4 else (page, 1)):
                raise ValueError("cache: each page must be contiguous")
    return _CacheArgument(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), of_k[0],
                          of_v[0], of_ks[0], of_vs[0], pages, heads, page, dim), device, heads, dim


def _within(t, strides):
    """Whether pages are contiguous but for dimensions of one element, whose strides say nothing."""
    return all(n == 1 or s == w for n, s, w in zip(t.shape[1:], t.stride()[1:], strides))


def _sequences(table, starts, lengths, device):
    """The C argument of a call's sequences."""
    size, of_starts, of_lengths = table.shape, starts.shape, lengths.shape
    if len(size) != 2 or len(of_starts) != 1 or len(of_lengths) != 1:
        raise ValueError("table is (sequences, most pages), starts (sequences + 1), lengths (sequences)")
    count, most = size
    if of_starts[0] != count + 1 or of_lengths[0] != count:
        raise ValueError(f"table names {count} sequences: starts must have {count + 1} entries and "
                         f"lengths {count}, not {of_starts[0]} and {of_lengths[0]}")
    row, column = table.stride()
    if not (table.dtype is _I32 and starts.dtype is _I32 and lengths.dtype is _I32
            and table.get_device() == device and starts.get_device() == device
            and lengths.get_device() == device and (column == 1 or most <= 1)
            and (starts.stride(0) == 1 or count == 0) and (lengths.stride(0) == 1 or count <= 1)):
        for name, t in (("table", table), ("starts", starts), ("lengths", lengths)):
            if t.dtype is not _I32:
                raise TypeError(f"{name}: expected torch.int32, got {t.dtype}")
            if t.get_device() != device:
                raise ValueError(f"{name}: every tensor must be on one CUDA device")
        raise ValueError("the entries of table's rows, of starts and of lengths must be contiguous")
    return _SequencesArgument(table.data_ptr(), row, most, starts.data_ptr(), lengths.data_ptr(), count)


def _rows(t, name, device, dtype, shape):
    """Pointer and element strides of a packed operand."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: every tensor must be on one CUDA device")
    token, head, element = t.stride()
    if element != 1:
        raise ValueError(f"{name}: a head's elements must be contiguous")
    return t.data_ptr(), token, head


def _rotation(rotate, dim):
    most = 6 if dim == 64 else 7
    if rotate is None:
        return most
    if not 0 <= rotate <= most:
        raise ValueError(f"rotate is 0 .. {most} for heads of {dim}")
    return rotate


def _packed(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name}: expected (tokens, heads, dim), got {t.dim()} dimensions")
    return t.shape


def _failed(status, what, operands):
    """The error of a call; says which operand does not start its rows on 16-byte boundaries."""
    if status == _fwt.FWT_ERR_MISALIGNED:
        for name, t in operands:
            size = t.element_size()
            apart = [s * size for s, n in zip(t.stride()[:2], t.shape) if n > 1]
            if t.data_ptr() % 16 or any(a % 16 for a in apart):
                what += (f": {name} starts at {t.data_ptr() % 16} bytes past a multiple of 16 and its rows "
                         f"are {apart} bytes apart")
                break
    return _fwt.FwtError(status, what)


def cache_append(k, v, cache, table, starts, lengths, rotate=None, stream=None):
    """Writes the new tokens' keys and values into their pages.

    ``k``, ``v``: (tokens, heads, dim), float32, bfloat16 or float16.  Each aligned group of
    ``2**rotate`` elements of a head (default: the whole head) is multiplied by the normalised H;
    the row gets the least power of two s with max|y| <= 448 s and codes e4m3(y / s).  A row that
    is not finite gets a NaN scale.  ``lengths`` count the new tokens.  Returns ``cache``."""
    if _lib is None:
        _load()
    held, device, heads, dim = _cache(cache)
    rotate = _rotation(rotate, dim)
    kind = _ff._REALS.get(k.dtype)
    if kind is None:
        raise TypeError(f"unsupported dtype {k.dtype}: use float32, bfloat16 or float16")
    shape = (_packed(k, "k")[0], heads, dim)
    at_k, at_v = _rows(k, "k", device, k.dtype, shape), _rows(v, "v", device, k.dtype, shape)
    places = _sequences(table, starts, lengths, device)
    st = _ff._run(device, stream, _lib.fwt_cache_append, *at_k, *at_v, kind, shape[0], held, places, rotate)
    if st != _fwt.FWT_OK:
        raise _failed(st, f"fwt_cache_append(tokens={shape[0]}, heads={heads}, dim={dim})",
                      [("k", k), ("v", v)])
    return cache


def cache_read(cache, table, starts, lengths, tokens: int, dtype=None, rotate=None, out=None, stream=None):
    """The last tokens of each sequence, scaled and turned back: (k, v), each (tokens, heads, dim)
    of ``dtype`` (bfloat16 by default, float16 or float32), or ``out``, a pair of tensors.

    ``tokens``: rows of the packed result, at least ``starts[-1]``; rows behind that are not
    written.  Rows without a token in the cache are zero."""
    if _lib is None:
        _load()
    held, device, heads, dim = _cache(cache)
    rotate = _rotation(rotate, dim)
    shape = (int(tokens), heads, dim)
    if out is None:
        dtype = dtype or _torch.bfloat16
        kind = _ff._REALS.get(dtype)
        if kind is None:
            raise TypeError(f"unsupported dtype {dtype}: use float32, bfloat16 or float16")
        k, v = _empty(shape, dtype, cache[0].device, stream), _empty(shape, dtype, cache[0].device, stream)
    else:
        k, v = out
        kind = _ff._REALS.get(k.dtype)
        if kind is None or (dtype is not None and k.dtype != dtype):
            raise TypeError(f"out: unsupported dtype {k.dtype}")
    at_k, at_v = _rows(k, "k", device, k.dtype, shape), _rows(v, "v", device, k.dtype, shape)
    places = _sequences(table, starts, lengths, device)
    st = _ff._run(device, stream, _lib.fwt_cache_read, held, places, rotate, *at_k, *at_v, kind, shape[0])
    if st != _fwt.FWT_OK:
        raise _failed(st, f"fwt_cache_read(tokens={shape[0]}, heads={heads}, dim={dim})", [("k", k), ("v", v)])
    return k, v


def _empty(shape, dtype, device, stream):
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _ff._allocations(device, stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def cache_attention(q, cache, table, starts, lengths, rotate=None, scale=None, causal: bool = True,
                    window: int = 0, longest: int = 0, out=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens, which the cache already holds, to all of it.

    ``q`` (tokens, q_heads, dim): bfloat16 or float16, q_heads a multiple of the cache's heads
    (consecutive query heads share one).  A token at position i sees the positions j below its
    sequence's length, with ``causal`` up to i, and with ``window`` > 0 only j > i - window; one that
    sees none gets zeros.  ``scale``: of the scores, 1/sqrt(dim) by default.  ``rotate``: as the
    cache was written.

    ``longest``: the most new tokens of any sequence as far as the caller knows, 0 as if all had
    the same; it chooses the kernel (whose roundings differ) and costs time where it is wrong.  ``out``: the tensor to
    write to.  ``workspace``: a CUDA tensor of ``fwt_cache_attention_workspace_bytes`` (allocated here
    when None), for one call at a time.  Returns out (tokens, q_heads, dim)."""
    if _lib is None:
        _load()
    held, device, heads, dim = _cache(cache)
    rotate = _rotation(rotate, dim)
    dtype = q.dtype
    kind = _ff._REALS.get(dtype)
    if kind != 1 and kind != 2:
        raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float16")
    shape = _packed(q, "q")
    tokens, q_heads, _ = shape
    if q_heads < 1 or q_heads % heads or shape[2] != dim:
        raise ValueError(f"q: {q_heads} heads of {shape[2]} for a cache of {heads} heads of {dim}")
    if window < 0 or longest < 0:
        raise ValueError("window and longest are 0 or more")
    at_q = _rows(q, "q", device, dtype, shape)
    places = _sequences(table, starts, lengths, device)
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
    at_out = _rows(out, "out", device, dtype, shape)
    longest = min(longest or -(-tokens // max(places.sequences, 1)), tokens)
    if workspace is None:
        size = _lib.fwt_cache_attention_workspace_bytes(q_heads, heads, dim, longest)
        workspace = _empty((size,), _torch.uint8, q.device, stream)
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        size = workspace.numel() * workspace.element_size()
    st = _ff._run(device, stream, _lib.fwt_cache_attention, *at_q, *at_out, kind, tokens, q_heads, held,
                  places, rotate, dim ** -0.5 if scale is None else scale, 1 if causal else 0, window,
                  longest, workspace.data_ptr(), size)
    if st != _fwt.FWT_OK:
        raise _failed(st, f"fwt_cache_attention(tokens={tokens}, heads={q_heads}/{heads}, dim={dim})",
                      [("q", q), ("out", out)])
    return out


def fwt_cache_attention_workspace_bytes(q_heads: int, heads: int, dim: int, longest: int) -> int:
    """Bytes of the workspace of ``cache_attention`` for sequences of up to ``longest`` new tokens."""
    return int(_fwt.library().fwt_cache_attention_workspace_bytes(q_heads, heads, dim, longest))
