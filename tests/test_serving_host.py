"""Serving operators without a GPU: the oracle's pins and the library's
refusals (each returns before any CUDA work)."""
import ctypes
import math
import os
import subprocess
import tempfile

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


# ---------------------------------------------------------------- oracle pins

def test_rotary_hand_case():
    """D = 4, rot = 4, theta = 100: w = 1, 0.1.  Position pi/2-like angles are
    not integers, so the frequencies are given: a quarter and a half turn."""
    w = np.array([math.pi / 2, math.pi])
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    half = S.rotary(x, [[1]], w)  # pairs (1, 3), (2, 4)
    assert np.allclose(half.ravel(), [-3, -2, 1, -4])
    inter = S.rotary(x, [[1]], w, layout="interleaved")  # pairs (1, 2), (3, 4)
    assert np.allclose(inter.ravel(), [-2, 1, -3, -4])
    back = S.rotary(half, [[1]], w, transpose=True)
    assert np.allclose(back, x)
    part = S.rotary(x, [[1]], w[:1])  # rot = 2: the rest passes
    assert np.allclose(part.ravel(), [-2, 1, 3, 4])


def test_rotary_gradient_against_differences():
    """The transposed rotation is the gradient of sum(g * y) by x."""
    rng = np.random.default_rng(3)
    x, g = rng.normal(size=(1, 2, 1, 6)), rng.normal(size=(1, 2, 1, 6))
    w = S.rotary_freqs(4, 100.0)
    pos = [[3, 1000]]
    grad = S.rotary(g, pos, w, "interleaved", 1.3, transpose=True)
    grad[..., 4:] = g[..., 4:]
    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-3
        num[i] = ((S.rotary(x + d, pos, w, "interleaved", 1.3) - S.rotary(x - d, pos, w, "interleaved", 1.3)) * g).sum() / 2e-3
    assert np.abs(grad - num).max() < 1e-9  # the map is linear: differences are exact up to rounding


def test_rotary_scalings():
    plain = S.rotary_freqs(64, 10000.0)
    assert np.allclose(plain[[0, 16]], [1.0, 0.01])
    assert np.allclose(S.rotary_freqs(64, 10000.0, "linear", 4.0), plain / 4)
    ntk = S.rotary_freqs(64, 10000.0, "ntk", 8.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], plain[-1] / 8)  # the last pair stretched by the factor
    for kind in ("turns", "ramp"):
        w = S.rotary_freqs(64, 10000.0, kind, 8.0, 4096)
        assert w[0] == plain[0] and np.isclose(w[-1], plain[-1] / 8)  # fast pairs kept, slow ones stretched
        assert np.all(np.diff(w / plain) <= 1e-15)


def test_prefix_decode_equals_one_softmax():
    """Two keys by hand: weights 2/3 and 1/3; an empty row; a prefix of one
    sequence only."""
    q = np.ones((3, 1, 1))
    K = np.full((3, 1, 2, 1), 50.0)
    V = np.full((3, 1, 2, 1), np.nan)
    K[0, 0, 0], V[0, 0, 0] = math.log(2.0), 3.0
    out, lse, w, _ = S.prefix_decode(q, K, V, [1, 0, 0], 1.0, np.zeros((1, 1, 1, 1)), np.full((1, 1, 1, 1), 6.0),
                                     [1], [0, 2], np.full((3, 1, 2), 0.5), 0.5)
    assert np.allclose(out.ravel(), [4.0, 6.0, 0.0])
    assert np.allclose(lse.ravel()[:2], [math.log(3.0), 0.0]) and lse[2, 0] == -np.inf
    assert np.allclose(w[0, 0], [0.25 + 2 / 3, 0.5]) and np.all(w[1:] == 0.5)


def test_cache_hand_cases():
    kept = S.cache_compress(np.array([[[9, 1, 3, 3, 0, 2.0]]]), [6], 4, 1, 1)
    assert kept == [[[0, 2, 3, 5]]]
    assert S.cache_compress(np.array([[[0, np.nan, 0, 0.0]]]), [4], 2, 0, 0) == [[[0, 2]]]
    assert S.cache_compress(np.array([[[5, 4, 3.0]]]), [2], 2, 0, 0) == [[[0, 1]]]
    c = dict(K=np.zeros((1, 1, 3, 1)), V=np.zeros((1, 1, 3, 1)), weights=np.array([[[1, 2, 1.0]]]),
             positions=np.array([[[4, 0, 2]]]), lengths=np.array([3]), next_pos=np.array([5]))
    one = np.ones((1, 1, 1))
    # position 0 is a sink, 4 is local: slot 2 is all that may go
    assert S.cache_insert(c, one, one, 3, 1, 1)[0, 0] == 2
    assert c["positions"].tolist() == [[[4, 0, 5]]] and c["weights"].tolist() == [[[1, 2, 0]]]
    assert c["next_pos"][0] == 6 and c["lengths"][0] == 3


# ---------------------------------------------------------------- layouts and refusals

@pytest.mark.parametrize("py,c", [("RotaryDesc", "csa_rotary_desc"), ("CacheDesc", "csa_cache_desc"),
                                  ("CacheSource", "csa_cache_source"),
                                  ("PrefixDecodeDesc", "csa_prefix_decode_desc")])
def test_descriptor_layouts(csa, py, c):
    """The ctypes mirrors have the C structs' sizes and field offsets."""
    cls = getattr(csa, py)
    fields = [f for f, _ in cls._fields_]
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "csa.h"', 'int main(void) {',
            f'  printf("%zu\\n", sizeof({c}));']
    prog += [f'  printf("%zu\\n", offsetof({c}, {f}));' for f in fields] + ['  return 0;', '}']
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(B.__file__))), "include")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        with open(src, "w") as f:
            f.write("\n".join(prog) + "\n")
        subprocess.run(["gcc", "-I", inc, src, "-o", exe], check=True)
        vals = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(cls)
    assert vals[1:] == [getattr(cls, f).offset for f in fields]


def test_rotary_pack_is_the_descriptor(csa):
    d = csa.RotaryDesc(1, 2, 3, (4, 5, 6), (7, 8, 9), 10, 11, 12, (13, 14, 15), (16, 17, 18), 1, 20, 21, 22, 23, 1, 1,
                       24, 2.5, 25, 26, -27)
    flat = csa.ROTARY_PACK.pack(1, 2, 3, *range(4, 10), 10, 11, 12, *range(13, 19), 1, 20, 21, 22, 23, 1, True, 24, 2.5,
                                25, 26, -27)
    e = csa.RotaryDesc.from_buffer_copy(flat)
    for f, _ in d._fields_:
        a, b = getattr(d, f), getattr(e, f)
        assert (list(a) == list(b)) if isinstance(a, ctypes.Array) else a == b, f


INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("change,status,word", [
    (dict(rot=3), INVALID, "rot"), (dict(rot=0), INVALID, "rot"), (dict(rot=130), INVALID, "rot"),
    (dict(D=127), INVALID, "D must be even"), (dict(D=1024, rot=64), UNSUPPORTED, "D must be"),
    (dict(layout=2), INVALID, "layout"), (dict(dtype=5), INVALID, "dtype"), (dict(B=-1), INVALID, "B"),
    (dict(amplitude=float("nan")), INVALID, "amplitude"), (dict(S=1 << 31), UNSUPPORTED, "2^29"),
    (dict(x_stride=(-128, 128, 128)), INVALID, "non-negative"),
    (dict(y_stride=(1024, 512, 64)), INVALID, "overlap"),
    (dict(layout=1, x_stride=(1025, 513, 129)), UNSUPPORTED, "even strides"),
    (dict(), INVALID, "x is NULL"),
])
def test_rotary_refusals(csa, change, status, word):
    kw = dict(B=2, S=2, H=4, D=128, rot=128, dtype=1, amplitude=1.0, x_stride=(1024, 512, 128),
              y_stride=(1024, 512, 128))
    kw.update(change)
    d = csa.rotary_desc(**kw)
    assert csa.lib.csa_rotary(ctypes.byref(d), None) == status
    assert word in csa.csa_last_error_string()


def test_rotary_table_refusals(csa):
    f = csa.lib.csa_rotary_table
    for args, word in [((3, 1e4, 0, 1.0, 1.0, 1.0, 2.0), "rot"), ((4, 1.0, 0, 1.0, 1.0, 1.0, 2.0), "theta"),
                       ((4, 1e4, 9, 1.0, 1.0, 1.0, 2.0), "scaling"), ((4, 1e4, 1, 0.5, 1.0, 1.0, 2.0), "factor"),
                       ((4, 1e4, 3, 2.0, 0.0, 1.0, 2.0), "orig_len"), ((4, 1e4, 3, 2.0, 9.0, 2.0, 2.0), "low"),
                       ((4, 1e4, 0, 1.0, 1.0, 1.0, 2.0), "table is NULL")]:
        assert f(*args, None, None, None) == INVALID
        assert word in csa.csa_last_error_string()
    assert csa.lib.csa_rotary(None, None) == INVALID


@pytest.mark.parametrize("change,status,word", [
    (dict(budget=0), INVALID, "budget"), (dict(budget=65), INVALID, "budget"), (dict(n_sink=-1), INVALID, "n_sink"),
    (dict(n_sink=32, n_local=32), INVALID, "below budget"), (dict(D=2048), UNSUPPORTED, "D must be"),
    (dict(T=1 << 31, budget=8), UNSUPPORTED, "T must be"), (dict(T=(1 << 31) - 65536, budget=8), UNSUPPORTED, "T must be"), (dict(B=1 << 15, Hkv=4), UNSUPPORTED, "65535"),
    (dict(dtype=9), INVALID, "dtype"), (dict(T=0), INVALID, "T positive"), (dict(), INVALID, "K is NULL"),
])
def test_cache_refusals(csa, change, status, word):
    kw = dict(dtype=1, B=1, Hkv=1, D=64, T=64, budget=64, k_stride=(4096, 4096, 64), v_stride=(4096, 4096, 64))
    kw.update(change)
    d = csa.cache_desc(**kw)
    two = (ctypes.c_int64 * 2)(64, 64)
    assert csa.lib.csa_cache_insert(ctypes.byref(d), None, two, None, two, None) == status
    assert word in csa.csa_last_error_string()
    if word != "below budget":  # compress: that budget is enough
        src = csa.cache_source(S=128)
        assert csa.lib.csa_cache_compress(ctypes.byref(d), ctypes.byref(src), None) == status


def test_compress_refusals(csa):
    d = csa.cache_desc(dtype=1, B=1, Hkv=1, D=64, T=64, budget=64, len=4096)
    for kw, status, word in [(dict(S=-1), INVALID, "S must be"), (dict(S=1 << 31), UNSUPPORTED, "S must be"), (dict(S=(1 << 31) - 65536), UNSUPPORTED, "S must be"),
                             (dict(S=8, positions=4096), INVALID, "next_pos"), (dict(S=8, len=4096), INVALID, "len")]:
        src = csa.cache_source(**kw)
        assert csa.lib.csa_cache_compress(ctypes.byref(d), ctypes.byref(src), None) == status
        assert word in csa.csa_last_error_string()
    assert csa.lib.csa_cache_compress(ctypes.byref(d), None, None) == INVALID
    assert csa.lib.csa_cache_insert(None, None, None, None, None, None) == INVALID


@pytest.mark.parametrize("change,status,word", [
    (dict(D=96), UNSUPPORTED, "D must be"), (dict(Hq=7), INVALID, "multiple"), (dict(Hq=34), UNSUPPORTED, "16"),
    (dict(N=65), UNSUPPORTED, "N must be"), (dict(B=1 << 16), UNSUPPORTED, "65535"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(scale=0.0), INVALID, "scale"),
    (dict(decay=-1.0), INVALID, "decay"), (dict(N=2), INVALID, "group_start"), (dict(out_dtype=4), INVALID, "out_dtype"),
    (dict(kp_stride=(8, 4, 128)), UNSUPPORTED, "Kp: strides"), (dict(kp_stride=(8, 8, 0)), UNSUPPORTED, "Kp: strides"), (dict(v_stride=(-8, 8, 128)), INVALID, "V: strides"),
    (dict(T=1 << 31), UNSUPPORTED, "Tp and T"), (dict(B=4096, T=1 << 30), UNSUPPORTED, "too many keys"),
    (dict(N=0, T=0), INVALID, "q is NULL"), (dict(), INVALID, "Kp is NULL"),
])
def test_prefix_decode_refusals(csa, change, status, word):
    kw = dict(dtype=1, B=2, Hq=8, Hkv=2, D=128, scale=0.1, N=1, Tp=128, T=64, decay=1.0)
    kw.update({f"{n}_stride": (0, 0, 128) for n in ("kp", "vp", "k", "v")})
    kw.update(change)
    d = csa.prefix_decode_desc(**kw)
    if word == "V: strides":  # the prefix's pointers come first
        d.N = 0
        d.K = None
    assert csa.lib.csa_prefix_decode(ctypes.byref(d), None) == status
    assert word in csa.csa_last_error_string()
    assert csa.lib.csa_prefix_decode(None, None) == INVALID


def test_binding_checks_tensors():
    """The classes refuse tensors whose layout the descriptors cannot say."""
    import torch
    from query_adaptive_chunk_b200 import csa, steps
    x = torch.zeros(2, 3, 4, 8)
    assert steps._rows("x", x.transpose(1, 2), torch.float32) == (96, 8, 32)
    for bad in (lambda: steps._rows("x", x.transpose(2, 3), torch.float32),
                lambda: steps._rows("x", x, torch.bfloat16),
                lambda: steps._dense("x", x.transpose(0, 1), torch.float32, (3, 2, 4, 8)),
                lambda: steps._dense("x", x, torch.float32, (2, 3, 4, 9)),
                lambda: steps._same_device(torch.device("cpu"), x=x.to("meta")),
                lambda: steps._typed("x", torch.float16), lambda: steps._empty_like(x, 5)):
        with pytest.raises(csa.CsaError):
            bad()
