"""Argument checks of the cache operators, all before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

import walsh_hadamard_transform_gb300 as fwt
from walsh_hadamard_transform_gb300 import build as fbuild
from walsh_hadamard_transform_gb300 import cache as fcache

A, GiB = 0x100000, 1 << 30  # fake, aligned addresses; validation never dereferences them
OK, E, MIS = fwt.FWT_OK, fwt.FWT_ERR_INVALID_ARG, fwt.FWT_ERR_MISALIGNED

PAGE = 2 * 32 * 64  # bytes of codes of a page
CACHE = dict(k=A, v=A + GiB, k_scale=A + 2 * GiB, v_scale=A + 3 * GiB, k_stride=PAGE, v_stride=PAGE,
             k_scale_stride=64, v_scale_stride=64, pages=10, heads=2, page_tokens=32, dim=64)
PLACES = dict(table=A + 4 * GiB, ld_table=5, most_pages=5, starts=A + 5 * GiB, lengths=A + 6 * GiB, sequences=3)
APPEND = dict(k=A + 7 * GiB, k_token=128, k_head=64, v=A + 8 * GiB, v_token=128, v_head=64,
              type=fwt.FWT_BF16, tokens=20, cache=CACHE, places=PLACES, rot=6, stream=None)
READ = dict(cache=CACHE, places=PLACES, rot=6, k=A + 7 * GiB, k_token=128, k_head=64, v=A + 8 * GiB,
            v_token=128, v_head=64, type=fwt.FWT_F32, tokens=20, stream=None)
ATTEND = dict(q=A + 7 * GiB, q_token=256, q_head=64, out=A + 8 * GiB, o_token=256, o_head=64,
              type=fwt.FWT_F16, tokens=20, q_heads=4, cache=CACHE, places=PLACES, rot=6, scale=0.125,
              causal=1, window=0, longest=0, ws=A + 9 * GiB, ws_bytes=1 << 29, stream=None)
ENTRY = {"append": ("fwt_cache_append", APPEND), "read": ("fwt_cache_read", READ),
         "attend": ("fwt_cache_attention", ATTEND)}

OF_CACHE = [
    (dict(dim=96), E), (dict(dim=256), E), (dict(heads=0), E), (dict(heads=65537), E), (dict(page_tokens=8), E),
    (dict(page_tokens=24), E), (dict(page_tokens=1 << 21), E), (dict(pages=-1), E), (dict(pages=1 << 31), E),
    (dict(heads=4096, page_tokens=1 << 20), E), (dict(k=None), E), (dict(v_scale=None), E), (dict(k_stride=PAGE - 16), E), (dict(v_scale_stride=48), E),
    (dict(k_stride=1 << 56), E), (dict(k=A + 8), MIS), (dict(v_scale=A + 3 * GiB + 4), MIS),
    (dict(v_stride=PAGE + 8), MIS), (dict(k_scale_stride=72), MIS),
]
OF_PLACES = [
    (dict(table=None), E), (dict(starts=None), E), (dict(lengths=None), E), (dict(sequences=-1), E),
    (dict(sequences=(1 << 30) + 1), E), (dict(most_pages=-1), E), (dict(most_pages=1 << 31), E), (dict(ld_table=4), E),
    (dict(ld_table=1 << 60), E), (dict(starts=A + 2), MIS), (dict(table=A + 1), MIS),
]
REFUSED = {
    "append": [
        (dict(type=3), E), (dict(type=-1), E), (dict(rot=7), E), (dict(rot=-1), E), (dict(tokens=-1), E),
        (dict(tokens=(1 << 30) + 1), E), (dict(k=None), E), (dict(v=None), E), (dict(k_token=-128), E),
        (dict(v_head=-64), E), (dict(v_token=1 << 41), E), (dict(k=A + 7 * GiB + 2), MIS), (dict(k_token=132), MIS),
        (dict(v_head=65), MIS), (dict(k=A), E), (dict(v=A + 2 * GiB), E),
        (dict(cache=dict(v=A)), E), (dict(cache=dict(k_scale=A + 64)), E), (dict(cache=dict(v=A + PAGE)), E),
    ],
    "read": [
        (dict(type=4), E), (dict(rot=7), E), (dict(tokens=-1), E), (dict(k=None), E), (dict(k_head=32), E),
        (dict(v_token=64), E), (dict(v=A + 8 * GiB + 4), MIS), (dict(k_token=130), MIS), (dict(v=A + 7 * GiB), E),
        (dict(v=A + 7 * GiB + 256), E), (dict(k=A + GiB), E),
    ],
    "attend": [
        (dict(type=fwt.FWT_F32), E), (dict(causal=2), E), (dict(window=-1), E), (dict(longest=-1), E),
        (dict(scale=float("inf")), E), (dict(scale=float("nan")), E), (dict(rot=7), E), (dict(q_heads=3), E),
        (dict(q_heads=0), E), (dict(q_heads=65538), E), (dict(tokens=-1), E), (dict(tokens=1 << 30), E),
        (dict(q=None), E), (dict(out=None), E), (dict(o_head=32), E), (dict(o_token=128), E),
        (dict(q=A + 7 * GiB + 8), MIS), (dict(o_token=260), MIS), (dict(ws=None), E), (dict(ws_bytes=1 << 10), E),
        (dict(ws=A + 9 * GiB + 8), MIS), (dict(out=A + 7 * GiB), E), (dict(out=A + 7 * GiB + 256), E),
        (dict(out=A), E), (dict(ws=A + 3 * GiB), E), (dict(ws=A + 8 * GiB), E), (dict(ws=A + 7 * GiB), E),
    ],
}


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fwt.library()


def call(entry, defaults, /, **changed):
    args = dict(defaults)
    assert not set(changed) - set(args)
    for name, kind in (("cache", fcache._CacheArgument), ("places", fcache._SequencesArgument)):
        args[name] = ctypes.byref(kind(**{**args[name], **changed.pop(name, {})}))
    args.update(changed)
    return entry(*args.values())


@pytest.mark.parametrize("which", sorted(REFUSED))
def test_refusals_before_any_launch(lib, which):
    name, defaults = ENTRY[which]
    changes = REFUSED[which] + [(dict(cache=c), st) for c, st in OF_CACHE] + [(dict(places=c), st) for c, st in OF_PLACES]
    for changed, status in changes:
        assert call(getattr(lib, name), defaults, **changed) == status, (name, changed)
    for struct in ("cache", "places"):
        args = {**defaults, "cache": ctypes.byref(fcache._CacheArgument(**CACHE)),
                "places": ctypes.byref(fcache._SequencesArgument(**PLACES)), struct: None}
        assert getattr(lib, name)(*args.values()) == E, (name, struct)


def test_empty_calls_need_no_gpu(lib):
    for which, (name, defaults) in ENTRY.items():
        nothing = {n: None for n in ("k", "v", "q", "out") if n in defaults}
        assert call(getattr(lib, name), defaults, tokens=0, **nothing) == OK, which
        assert call(getattr(lib, name), defaults, places=dict(sequences=0, table=None, starts=None, lengths=None),
                    **nothing) == OK, which
    empty = dict(pages=0, k=None, v=None, k_scale=None, v_scale=None)
    assert call(lib.fwt_cache_append, APPEND, cache=empty) == OK
    assert call(lib.fwt_cache_append, APPEND, places=dict(most_pages=0, table=None)) == OK


def test_windows_side_by_side_are_no_overlap(lib):
    """Those calls pass every check: with no tokens' sequences to look at, nothing is launched."""
    # a pool of pages that hold keys, values and their scales one after the other
    pool = dict(v=A + PAGE, k_scale=A + 2 * PAGE, v_scale=A + 2 * PAGE + 64)
    pitch = {n: 2 * PAGE + 128 for n in ("k_stride", "v_stride", "k_scale_stride", "v_scale_stride")}
    missing = dict(places=dict(starts=A + 1))  # refused last, for its alignment
    assert call(lib.fwt_cache_append, APPEND, cache={**pool, **pitch}, **missing) == MIS
    assert call(lib.fwt_cache_append, APPEND, cache={**pool, **pitch, "v": A + PAGE - 16}, places={}) == E
    # keys and values of one output tensor
    assert call(lib.fwt_cache_read, READ, v=A + 7 * GiB + 512, k_token=256, v_token=256, **missing) == MIS
    assert call(lib.fwt_cache_read, READ, v=A + 7 * GiB + 496, k_token=256, v_token=256) == E


def test_workspace_size(lib):
    size = lib.fwt_cache_attention_workspace_bytes
    assert size(8, 8, 128, 1) >= 192 * 2 * 8 * 130 * 4
    assert size(8, 8, 128, 0) == size(8, 8, 128, 1) <= size(8, 8, 128, 3000)
    assert size(8, 3, 128, 1) == size(0, 1, 128, 1) == size(8, 8, 96, 1) == size(8, 8, 128, -1) == 0
    assert fwt.fwt_cache_attention_workspace_bytes(8, 8, 128, 1) == size(8, 8, 128, 1)


def test_binding_checks():
    cache = fwt.new_cache(3, 16, 2, 64, device="cpu")
    assert cache.k.shape == (3, 2, 16, 64) and cache.v_scale.shape == (3, 2, 16)
    assert cache.k.dtype == torch.float8_e4m3fn and cache.k_scale.dtype == torch.float8_e8m0fnu
    for bad in ((3, 16, 2, 96), (3, 24, 2, 64), (3, 8, 2, 64), (3, 16, 0, 64), (-1, 16, 2, 64)):
        with pytest.raises(ValueError, match="page_tokens"):
            fwt.new_cache(*bad, device="cpu")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for f in (lambda c: fwt.cache_append(x, x, c, *i), lambda c: fwt.cache_read(c, *i, 4),
              lambda c: fwt.cache_attention(x, c, *i)):
        with pytest.raises(ValueError, match="CUDA device"):
            f(cache)
        with pytest.raises(ValueError, match="codes are"):
            f(cache._replace(v=cache.v[:2]))
        with pytest.raises(ValueError, match="scales are"):
            f(cache._replace(v_scale=cache.v_scale[:, :1]))
        with pytest.raises(TypeError, match="float8"):
            f(cache._replace(k=cache.k.view(torch.uint8)))
        with pytest.raises(ValueError, match="dim is 64 or 128"):
            f(fwt.Cache(*(t[..., :32] if t.dim() == 4 else t for t in cache)))


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(fcache._CacheArgument) == 4 * 8 + 5 * 8 + 3 * 4 + 4
    assert ctypes.sizeof(fcache._SequencesArgument) == 6 * 8
