"""Serving operators on the GPU: states and calls that an ordinary batch does
not have (paused sequences, positions at the end of their range, gradients
through autograd, refused steps), against the fp64 oracle or the exact values."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as S
from oracle.pipeline import to_np

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def csa():
    from query_adaptive_chunk_b200 import csa as mod
    return mod


@pytest.fixture(scope="module")
def steps():
    from query_adaptive_chunk_b200 import steps as mod
    return mod


def _randn(shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- paused sequences

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,prefixes", [(4, 1), (4, 0), (12, 1), (2, 2)])
def test_step_leaves_a_paused_sequence_alone(steps, csa, dtype, G, prefixes):
    """A negative next position: no key enters, the sums stay as they are (whatever
    the unused query and key rows hold), out = 0 and lse = -inf; the others
    get what they get without it.  Unpaused, it goes on where it was."""
    B, Hkv, D, T, Tp = 6, 2, 64, 70, 150
    dt = DT[dtype]
    Kp, Vp = _randn((max(1, prefixes), Hkv, Tp, D), 1, dt), _randn((max(1, prefixes), Hkv, Tp, D), 2, dt)
    kw = {}
    if prefixes:
        kw = dict(Kp=Kp, Vp=Vp, group_start=_i32([0, 4] if prefixes == 1 else [0, 2, 5]))
    K, V = _randn((B, Hkv, T, D), 3, dt), _randn((B, Hkv, T, D), 4, dt)
    q, k, v = (_randn((B, n, D), 5 + n, dt) for n in (Hkv * G, Hkv, Hkv))
    paused = [1, 5]

    def run(pause):
        cache = steps.TokenCache(K.clone(), V.clone(), lengths=_i32([T, 40, 0, 1, 69, T]), n_local=3,
                                 next_pos=_i32([T, 40, 0, 1, 69, T]), positions=torch.arange(T, dtype=torch.int32, device="cuda").expand(B, Hkv, T).contiguous(),
                                 weights=_randn((B, Hkv, T), 9).argsort(-1).float() + 1)  # far apart
        before = {n: getattr(cache, n).clone() for n in ("K", "V", "weights", "positions", "lengths")}
        dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, decay=0.5, rotary=steps.Rotary(32), **kw)
        held = cache.next_pos.clone()
        qs, ks = q.clone(), k.clone()
        if pause:
            cache.next_pos[paused] = -7
            qs[paused], ks[paused] = float("nan"), float("nan")
        for _ in range(2):
            out, lse = dec.step(qs, ks, v)
            csa.csa_check_device_status()
        got = out.clone(), lse.clone(), cache.weights.clone(), cache.K.clone(), cache.lengths.clone(), cache.positions.clone()
        if not pause:
            return got
        assert cache.next_pos[paused].tolist() == [-7, -7]
        for n, x in before.items():
            assert torch.equal(getattr(cache, n)[paused], x[paused]), n
        assert not out[paused].any() and bool((lse[paused] == -math.inf).all())
        cache.next_pos[paused] = held[paused]
        for _ in range(2):
            out, lse = dec.step(q, k, v)
        csa.csa_check_device_status()
        return got, (out.clone(), lse.clone(), cache.weights.clone())

    want = run(False)
    got, later = run(True)
    others = [b for b in range(B) if b not in paused]
    # Without the paused sequences' keys the split of the others' is another, and so is the
    # order of their sums: a logit and the running sums are good to 2^-20 + 2 * 68 * 2^-24
    # sum |q k| / 8 < 1e-4 of a weight, an output to that and to bf16's rounding of the
    # weights; two runs of two steps of G <= 12 weights each.
    u = U16 if dtype == "bf16" else 0.0
    vmax = float(max(V.abs().max(), v.abs().max(), Vp.abs().max()))
    for rows, (o, l, w) in ((others, got[:3]), (paused, later)):
        assert float((o[rows] - want[0][rows]).abs().max()) <= 2 * (1e-4 + u) * vmax
        assert float((l[rows] - want[1][rows]).abs().max()) <= 2e-4
        assert float((w[rows] - want[2][rows]).abs().max()) <= 2 * 2 * 12 * 1e-4
    for x, y in zip(got[3:], want[3:]):
        assert torch.equal(x[others], y[others])


def test_attend_takes_a_paused_batch(steps, csa):
    """Every sequence paused: nothing but zeros and -inf, the sums as they were."""
    K = _randn((3, 2, 40, 128), 1, torch.bfloat16)
    cache = steps.TokenCache(K, K.clone(), lengths=_i32([40, 3, 0]), next_pos=_i32([-1, -2, -(1 << 31)]),
                             weights=_randn((3, 2, 40), 2))
    before = cache.weights.clone()
    Kp = _randn((1, 2, 300, 128), 3, torch.bfloat16)
    dec = steps.SharedPrefixDecoder(cache, Hq=8, Kp=Kp, Vp=Kp, decay=0.0)
    out, lse = dec.attend(_randn((3, 8, 128), 4, torch.bfloat16))
    csa.csa_check_device_status()
    assert not out.any() and bool((lse == -math.inf).all()) and torch.equal(cache.weights, before)


@pytest.mark.parametrize("B,Hkv,Sn,T,n_sink,n_local", [
    (3, 2, 100, 33, 4, 8), (2, 1, 4097, 1000, 4, 100), (1, 2, 20000, 513, 0, 300), (20, 8, 9000, 31, 2, 29),
    (3, 1, 70001, 300, 8, 292), (2, 1, 400003, 64, 3, 17), (2, 2, 50, 20, 0, 0)])
def test_compress_of_paused_sequences(steps, csa, B, Hkv, Sn, T, n_sink, n_local):
    """A paused sequence's cache is compressed as another's: its sinks, the rows of its last
    positions and the heaviest others stay, and so does the pause."""
    rng = np.random.default_rng(Sn)
    D = 6
    w = rng.random((B, Hkv, Sn)).astype(np.float32)
    pos = np.argsort(rng.random((B, Hkv, Sn)), -1) * 2 + 1
    n = rng.integers(Sn // 2, Sn + 1, B)
    n[0] = Sn
    nxt = np.full(B, 2 * Sn + 5)
    nxt[::2] = [-1 - (b * (1 << 31) // (2 * B)) for b in range(0, B, 2)]
    nxt[0] = -(1 << 31)
    K = _randn((B, Hkv, Sn, D), 3)
    for given in (False, True):
        cache = steps.TokenCache(torch.zeros(B, Hkv, T, D, device="cuda"), torch.zeros(B, Hkv, T, D, device="cuda"),
                                 n_sink=n_sink, n_local=n_local)
        cache.compress(K, K, torch.tensor(w, device="cuda"), lengths=_i32(n.tolist()), next_pos=_i32(nxt.tolist()),
                       positions=_i32(pos.tolist()) if given else None)
        csa.csa_check_device_status()
        kept = S.cache_compress(w, n, T, n_sink, n_local, pos if given else None, nxt)
        assert cache.next_pos.tolist() == nxt.tolist()
        for b in range(B):
            for h in range(Hkv):
                rows = kept[b][h]
                assert cache.lengths[b] == len(rows)
                want = pos[b, h, rows] if given else rows
                assert cache.positions[b, h, :len(rows)].tolist() == list(want)
                assert torch.equal(cache.K[b, h, :len(rows)], K[b, h, rows])


def test_compress_within_one_buffer(steps, csa):
    """The cache is the first slots of each unit's storage, the source the others."""
    B, Hkv, T, Sn, D = 3, 2, 20, 90, 64
    K, V = _randn((B, Hkv, T + Sn, D), 1, torch.bfloat16), _randn((B, Hkv, T + Sn, D), 2, torch.bfloat16)
    w = torch.rand(B, Hkv, Sn, device="cuda")
    Ks, Vs = K[:, :, T:], V[:, :, T:]
    source = Ks.clone(), Vs.clone()
    cache = steps.TokenCache(K[:, :, :T], V[:, :, :T], n_sink=2, n_local=5, next_pos=_i32([Sn, 40, 3]))
    cache.compress(Ks, Vs, w, lengths=cache.next_pos)
    csa.csa_check_device_status()
    assert cache.next_pos.tolist() == [Sn, 40, 3] and cache.lengths.tolist() == [T, T, 3]
    kept = S.cache_compress(to_np(w), [Sn, 40, 3], T, 2, 5)
    for b in range(B):
        for h in range(Hkv):
            rows = kept[b][h]
            assert cache.positions[b, h, :len(rows)].tolist() == rows
            for x, s in ((K, source[0]), (V, source[1])):
                assert torch.equal(x[b, h, :len(rows)], s[b, h, rows])
    assert torch.equal(K[:, :, T:], source[0]) and torch.equal(V[:, :, T:], source[1])
