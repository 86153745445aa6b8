"""Serving operators without a GPU: refusals and oracle pins of states that an
ordinary batch does not have (each refusal returns before any CUDA work)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import serving as S
from query_adaptive_chunk_b200 import build as B


@pytest.fixture(scope="module")
def csa():
    if not os.path.exists(B.LIB) or any(os.path.getmtime(s) > os.path.getmtime(B.LIB)
                                        for s in B.sources()):
        B.build()
    from query_adaptive_chunk_b200 import csa as mod
    return mod


INVALID, UNSUPPORTED = 1, 2


def test_compress_of_a_paused_sequence_by_hand():
    """Position 9 is the last one, so 8 and 9 are local; 3 is the heaviest other."""
    w = np.array([[[0.0, 5.0, 1.0, 0.0, 2.0]]])
    pos = np.array([[[8, 3, 4, 9, 5]]])
    assert S.cache_compress(w, [5], 3, 0, 2, pos, [-1]) == [[[0, 1, 3]]]
    assert S.cache_compress(w, [5], 3, 0, 2, pos, [10]) == [[[0, 1, 3]]]
    assert S.cache_compress(w, [5], 3, 0, 2, None, [-1]) == [[[1, 3, 4]]]


def _cache(csa, **kw):
    d = dict(dtype=1, B=2, Hkv=4, D=64, T=32, budget=32, K=1 << 20, V=1 << 30, k_stride=(8192, 2048, 64),
             v_stride=(8192, 2048, 64))
    d.update(kw)
    return csa.cache_desc(**d)


def _insert(csa, d, k, k_stride, v, v_stride):
    two = ctypes.c_int64 * 2
    status = csa.lib.csa_cache_insert(ctypes.byref(d), ctypes.c_void_p(k), two(*k_stride), ctypes.c_void_p(v),
                                      two(*v_stride), None)
    return status, csa.csa_last_error_string()


K0, V0, FREE = 1 << 20, 1 << 30, 1 << 40  # addresses that nothing reads: each call is refused before


def test_insert_refuses_rows_of_the_cache(csa):
    """New rows out of the cache itself could be read after their slot was written."""
    d = _cache(csa)
    row = (256, 64)
    slot0 = (8192, 2048)  # slot 0 of each unit, as a view
    for k, ks, v, vs in [(K0, slot0, FREE, row), (FREE, row, V0, slot0), (V0, slot0, FREE, row),
                         (K0 + 2 * 64 * 31, slot0, FREE, row), (K0, (0, 0), FREE, row),
                         (K0 - 2, row, FREE, row)]:
        status, why = _insert(csa, d, k, ks, v, vs)
        assert status == INVALID and "overlap" in why, why
    # beside the cache, and in the same buffer between its rows (a slot that is not the cache's)
    between = _cache(csa, T=31, budget=31)
    for dd, k, ks in [(d, K0 + 2 * 64 * 32 * 8, row), (d, K0 - 2 * 64 * 8, row), (between, K0 + 2 * 64 * 31, slot0)]:
        status, why = _insert(csa, dd, k, ks, FREE, row)
        assert "overlap" not in why, why  # (refused later on: no such memory)


def test_cache_refuses_slots_that_overlap(csa):
    for kw in (dict(k_stride=(64, 2048, 64)), dict(v_stride=(2048, 2048, 64)), dict(k_stride=(0, 2048, 64)),
               dict(V=K0), dict(V=K0 + 2 * 64 * 32 * 4), dict(V=K0 + 126)):
        d = _cache(csa, **kw)
        status, why = _insert(csa, d, FREE, (256, 64), FREE, (256, 64))
        assert status == INVALID and "overlap" in why, (kw, why)
        src = csa.cache_source(S=0)
        assert csa.lib.csa_cache_compress(ctypes.byref(d), ctypes.byref(src), None) == INVALID
        assert "overlap" in csa.csa_last_error_string(), kw
    # K and V in one buffer, a slot's key and value side by side
    d = _cache(csa, V=K0 + 128, k_stride=(16384, 4096, 128), v_stride=(16384, 4096, 128))
    assert "overlap" not in _insert(csa, d, FREE, (256, 64), FREE, (256, 64))[1]


def _rotary(csa, **kw):
    d = dict(B=2, S=5, H=4, H2=2, D=64, rot=32, dtype=1, amplitude=1.0, x=K0, y=V0, x2=FREE, y2=FREE + (1 << 20))
    d.update({f"{t}_stride": (5 * 256, 256, 64) for t in ("x", "y")})
    d.update({f"{t}_stride": (5 * 128, 128, 64) for t in ("x2", "y2")})
    d.update(kw)
    status = csa.lib.csa_rotary(ctypes.byref(csa.rotary_desc(**d)), None)
    return status, csa.csa_last_error_string()


def test_rotary_refuses_outputs_over_other_rows(csa):
    """A thread's row could be written before another thread reads it."""
    head = 2 * 64
    packed = dict(x=K0, x2=K0 + 4 * head, x_stride=(5 * 512, 512, 64), x2_stride=(5 * 512, 512, 64))
    for kw in (dict(y=K0 + head),                                   # a head further on in its own input
               dict(y=K0 + 2), dict(y=K0 - 2),
               dict(y=K0, y_stride=(5 * 256, 256 // 4, 5 * 64)),    # in place in another order
               dict(x2=V0), dict(y2=K0), dict(y2=V0),               # over the other tensor
               dict(packed, y=K0 + 4 * head, y_stride=(5 * 512, 512, 64)),
               dict(y_stride=(64, 64, 64)), dict(y2_stride=(128, 128, 64)),  # rows of one output
               dict(x2=K0, x2_stride=(5 * 256, 256, 64), y=K0)):    # turned in place and read besides
        status, why = _rotary(csa, **kw)
        assert status == INVALID and "overlap" in why, (kw, why)
    own = dict(packed, y=K0, y2=K0 + 4 * head, y_stride=(5 * 512, 512, 64), y2_stride=(5 * 512, 512, 64))
    for kw in ({}, own, dict(packed, y=K0, y_stride=(5 * 512, 512, 64)), dict(x_stride=(0, 256, 64)),
               dict(x2=K0), dict(packed, y=K0 + 6 * head, x_stride=(5 * 1024, 1024, 64), x2_stride=(5 * 1024, 1024, 64),
                                 y_stride=(5 * 1024, 1024, 64))):
        status, why = _rotary(csa, **kw)
        assert "overlap" not in why, (kw, why)  # (refused later on: no such memory)


def _compress(csa, d, **kw):
    src = dict(S=40, K=FREE, V=FREE + (1 << 24), k_stride=(4 * 40 * 64, 40 * 64, 64), v_stride=(4 * 40 * 64, 40 * 64, 64),
               weights=FREE + (1 << 25))
    src.update(kw)
    s = csa.cache_source(**src)
    status = csa.lib.csa_cache_compress(ctypes.byref(d), ctypes.byref(s), None)
    return status, csa.csa_last_error_string()


def test_compress_takes_rows_beside_the_cache(csa):
    """One buffer of 72 slots a unit: the first 32 are the cache, the rest the source."""
    unit = 72 * 64
    st = (4 * unit, unit, 64)
    d = _cache(csa, k_stride=st, v_stride=st)
    beside = dict(K=K0 + 32 * 128, V=V0 + 32 * 128, k_stride=st, v_stride=st)
    assert "overlap" not in _compress(csa, d, **beside)[1]
    for kw in (dict(beside, K=K0 + 31 * 128), dict(beside, V=V0 + 32 * 128 - 2), dict(beside, V=K0), dict(beside, S=41)):
        status, why = _compress(csa, d, **kw)
        assert status == INVALID and "overlap" in why, kw


def test_compress_refuses_lengths_that_it_writes(csa):
    """Every head reads the source's length and one of them writes the cache's state."""
    L, P = 1 << 41, 1 << 42
    d = _cache(csa, B=8, Hkv=1, len=L, next_pos=P, k_stride=(2048, 2048, 64), v_stride=(2048, 2048, 64))
    free = 1 << 43
    for kw, word in [(dict(len=L), "len"), (dict(len=L + 16), "len"), (dict(next_pos=L), "next_pos"), (dict(next_pos=P - 16), "next_pos"),
                     (dict(len=P, next_pos=free), "next_pos"), (dict(len=P + 16), "next_pos")]:
        status, why = _compress(csa, d, **kw)
        assert status == INVALID and word in why and "CUDA" not in why, (kw, why)
    for kw in (dict(len=P), dict(next_pos=P), dict(len=free, next_pos=P), dict(len=L + 32, next_pos=P + 32)):
        assert "CUDA" in _compress(csa, d, **kw)[1], kw  # goes on to the pointers


def test_strides_of_single_entries_are_not_used(csa):
    """Views leave odd or no strides where an index has one entry; each call goes on
    to its pointers."""
    status, why = _rotary(csa, B=1, S=1, H2=0, layout=1, x_stride=(7, 5, 64), y_stride=(3, 0, 64))
    assert "CUDA" in why, why
    status, why = _rotary(csa, B=1, S=5, H=1, H2=0, x_stride=(-1, 128, 9), y_stride=(1, 128, 77))
    assert "CUDA" in why, why
    status, why = _rotary(csa, B=1, S=5, H=1, H2=0, x_stride=(5, 128, 3), y_stride=(9, 128, 0), y=K0)  # in place
    assert "CUDA" in why, why
    d = _cache(csa, B=1, Hkv=1, k_stride=(1, 3, 64), v_stride=(0, -5, 64))
    assert "CUDA" in _insert(csa, d, FREE, (-1, 3), FREE, (0, 1))[1]
    assert "CUDA" in _compress(csa, d, k_stride=(-1, 3, 64), v_stride=(1, 0, 64))[1]
    two = dict(k_stride=(31, 33, 128), v_stride=(-2, 1, 128), kp_stride=(5, 7, 128), vp_stride=(-1, 0, 128))
    kw = dict(dtype=1, B=1, Hq=4, Hkv=1, D=128, scale=0.1, N=1, Tp=128, T=64, decay=1.0, K=K0, V=V0, Kp=FREE, Vp=FREE, **two)
    for change, word in [({}, "CUDA"), (dict(Tp=1, T=1, k_stride=(1, 1, 1), kp_stride=(1, 1, 1)), "CUDA"),
                         (dict(B=2, N=0), "V: strides"), (dict(Hkv=2), "Kp: strides")]:
        d = csa.prefix_decode_desc(**{**kw, **change})
        if "V" in word:
            d.k_stride = (ctypes.c_int64 * 3)(64 * 128, 1, 128)
        assert csa.lib.csa_prefix_decode(ctypes.byref(d), None) in (INVALID, UNSUPPORTED)
        assert word in csa.csa_last_error_string(), change


@pytest.mark.parametrize("missing", ["_raw_stream", "_device"])
def test_current_stream_by_torchs_public_call(csa, monkeypatch, missing):
    """A torch without the two short cuts still gives the current stream."""
    import types

    import torch
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x1230))
    monkeypatch.setattr(csa, missing, None)
    assert csa._s(None).value == 0x1230
    assert csa._s(0x77).value == 0x77
