"""Serving operators on the GPU against the fp64 oracle: rotary positions, the
decode over shared prefixes, the cache bounded by attention weight, and a run of
them together.

Tolerances.  u = eps / 2 is a rounding's relative error (bf16 2^-8, fp32
2^-24).  Rotary: the angle as a float in half turns is off by u * pi radians,
sincospif by two steps, the amplitude, two products and a sum by u each: less
than 10 u (2^-24) of A (|x_a| + |x_b|) < 6e-7, then the result's rounding.
Decode: a logit is a sum of D products, off by at most (D + 4) u of its
absolute sum (call the largest E, in nats); the running maximum and sum add
2^-20 (ex2.approx is good to 2^-22).  A weight p_j is then off by 2 E + 2^-20 of
itself, so is out's error against sum p_j |v_j|, to which bf16 adds the
rounding of p_j (2^-8) and the output's own."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as S
from oracle.serving import rotary_freqs as oracle_freqs
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


# ---------------------------------------------------------------- rotary

def _rotary_close(got, x, pos, freqs, layout, amp, transpose):
    want = S.rotary(to_np(x), pos, freqs, layout, amp, transpose)
    u = U16 if x.dtype == torch.bfloat16 else U32
    size = S.rotary(np.abs(to_np(x)), np.zeros_like(pos), freqs, layout, 1.0)
    rot = 2 * len(freqs)
    other = np.array(size)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    other[..., a], other[..., b] = size[..., b], size[..., a]
    tol = u * np.abs(want) + 6e-7 * abs(amp) * (size + other)
    err = np.abs(got.cpu().double().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()
    assert np.array_equal(to_np(got)[..., rot:], to_np(x)[..., rot:])  # the rest is copied


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Sq,Hq,Hkv,D,rot", [(1, 1, 1, 1, 64, 64), (3, 1, 32, 8, 128, 128), (2, 37, 7, 1, 128, 64),
                                               (1, 129, 4, 2, 80, 20), (2, 5, 3, 3, 96, 24), (1, 3, 2, 1, 6, 2),
                                               (1, 300, 16, 16, 256, 256), (2, 2, 5, 1, 512, 6)])
def test_rotary_shapes(steps, dtype, layout, B, Sq, Hq, Hkv, D, rot):
    q, k = _randn((B, Sq, Hq, D), 1, DT[dtype]), _randn((B, Sq, Hkv, D), 2, DT[dtype])
    rng = np.random.default_rng(B * 100 + D)
    pos = rng.integers(0, 1 << 20, (B, Sq))
    pos[0, 0] = 0
    r = steps.Rotary(rot, theta=10000.0, layout=layout, amplitude=1.25)
    w = S.rotary_freqs(rot, 10000.0)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for t in (False, True):
        yq, yk = r.rotate(q, k, positions=p, transpose=t)
        _rotary_close(yq, q, pos, w, layout, 1.25, t)
        _rotary_close(yk, k, pos, w, layout, 1.25, t)


@pytest.mark.parametrize("kind,factor,orig", [("none", 1.0, 1), ("linear", 4.0, 1), ("ntk", 8.0, 1), ("turns", 8.0, 8192),
                                              ("ramp", 32.0, 4096), ("ramp", 2.0, 3), ("turns", 1.0, 2048)])
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000.0), (2, 10000.0)])
def test_rotary_scalings_far(steps, kind, factor, orig, rot, theta):
    """Every frequency rule, at positions up to the last int32 and below zero."""
    pos = np.array([[0, 1, 8191, 131071, 1 << 20, (1 << 31) - 1, -1, -(1 << 31)]])
    x = _randn((1, 8, 2, 128), 5)
    r = steps.Rotary(rot, theta=theta, scaling=kind, factor=factor, orig_len=orig)
    y = r.rotate(x, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    w = S.rotary_freqs(rot, theta, kind, factor, orig)
    # the oracle's own angle is off by u64 * p w (and its frequency by a few u64): only
    # 2^31 * 2^-51 = 1e-6 rad at the far ends
    want = S.rotary(to_np(x), pos, w)
    err = np.abs(to_np(y) - want)
    far = np.abs(pos[0]) > 1 << 21
    size = np.abs(to_np(x)).max()
    assert err[:, ~far].max() <= 2 * size * 6e-7 + U32 * size
    assert err[:, far].max() <= 2 * size * 5e-6


def test_rotary_own_frequencies(steps):
    w = torch.rand(16, dtype=torch.float64, device="cuda") * 20 - 10  # several turns a position, either way
    x = _randn((1, 50, 3, 64), 6)
    y = steps.Rotary(32, freqs=w).rotate(x, pos0=1000)
    _rotary_close(y, x, np.arange(1000, 1050)[None], w.cpu().numpy(), "half", 1.0, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_views_in_place_and_odd_strides(steps, dtype):
    """Packed projections, head-major outputs, broadcast positions, in place,
    rows that start off 16 bytes, a stream of its own."""
    B, Sq, Hq, Hkv, D = 2, 33, 6, 2, 64
    packed = _randn((B, Sq, (Hq + 2 * Hkv) * D), 7, DT[dtype])
    q, k = packed[..., :Hq * D].view(B, Sq, Hq, D), packed[..., Hq * D:(Hq + Hkv) * D].view(B, Sq, Hkv, D)
    cache = torch.zeros(B, Hkv, 50, D, dtype=DT[dtype], device="cuda")
    r = steps.Rotary(32, theta=10000.0)
    w = S.rotary_freqs(32, 10000.0)
    pos = np.tile(np.arange(100, 100 + Sq), (B, 1))
    p = torch.arange(100, 100 + Sq, dtype=torch.int32, device="cuda")[None].expand(B, Sq)
    v0 = packed[..., (Hq + Hkv) * D:].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.rotate(q, k, positions=p, k_out=cache[:, :, 7:7 + Sq].transpose(1, 2), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _rotary_close(cache[:, :, 7:7 + Sq].transpose(1, 2), k, pos, w, "half", 1.0, False)
    assert not cache[:, :, :7].any() and not cache[:, :, 7 + Sq:].any()
    before = q.clone()
    r.rotate(q, q_out=q, pos0=100)
    _rotary_close(q, before, pos, w, "half", 1.0, False)
    assert torch.equal(packed[..., (Hq + Hkv) * D:], v0)
    odd = _randn((B, Sq, 3, D + 1), 8, DT[dtype])[..., :D]  # rows D + 1 apart
    _rotary_close(r.rotate(odd, pos0=100), odd, pos, w, "half", 1.0, False)
    even = _randn((B, Sq, 3, D + 2), 9, DT[dtype])[..., :D]
    _rotary_close(steps.Rotary(32, layout="interleaved").rotate(even, pos0=100), even, pos, w, "interleaved", 1.0, False)


def test_rotary_refuses(csa, steps):
    r = steps.Rotary(64)
    x = torch.zeros(1, 4, 2, 128, device="cuda")
    with pytest.raises(csa.CsaError):
        r.rotate(x, positions=torch.zeros(1, 4, device="cuda"))  # not int32
    with pytest.raises(csa.CsaError):
        r.rotate(x, positions=torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(csa.CsaError):
        r.rotate(x[..., :32])  # narrower than rot
    with pytest.raises(csa.CsaError):
        r.rotate(x.transpose(-1, -2))
    with pytest.raises(csa.CsaError):
        r.rotate(x.cpu())
    assert r.rotate(x[:, :0]).shape == (1, 0, 2, 128)  # nothing to do


# ---------------------------------------------------------------- cache

def _cache_state(B, Hkv, T, D, dtype, seed, full=True, ties=False):
    g = np.random.default_rng(seed)
    w = g.random((B, Hkv, T)).astype(np.float32)
    if ties:
        w = np.floor(w * 4).astype(np.float32)
        w[:, :, ::7] = -0.0
        w[:, :, 3::11] = np.nan
        w[:, :, 5::13] = -np.inf
        w[:, :, 6::17] = np.inf
    pos = np.argsort(g.random((B, Hkv, T)), -1) * 2
    n = np.full(B, T) if full else g.integers(0, T + 1, B)
    return dict(K=_randn((B, Hkv, T, D), seed, dtype), V=_randn((B, Hkv, T, D), seed + 1, dtype),
                weights=torch.tensor(w, device="cuda"), positions=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                lengths=torch.tensor(n, dtype=torch.int32, device="cuda"),
                next_pos=torch.tensor(np.full(B, 2 * T), dtype=torch.int32, device="cuda"))


def _host(state):
    return {k: (to_np(v) if v.dtype.is_floating_point else v.cpu().numpy().copy()) for k, v in state.items()}


def _same(state, want):
    for k, v in state.items():
        got = to_np(v) if v.dtype.is_floating_point else v.cpu().numpy()
        assert np.array_equal(got, want[k], equal_nan=got.dtype.kind == "f"), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,T,D,n_sink,n_local,ties,full", [
    (1, 1, 1, 64, 0, 0, False, True), (2, 3, 33, 64, 4, 8, True, True), (3, 1, 513, 96, 0, 1, True, True),
    (2, 2, 2049, 128, 4, 100, False, True), (4, 2, 65, 80, 2, 3, True, False), (2, 1, 5000, 6, 1, 64, True, True)])
def test_cache_insert(steps, csa, dtype, B, Hkv, T, D, n_sink, n_local, ties, full):
    s = _cache_state(B, Hkv, T, D, DT[dtype], T + D, full, ties)
    want = _host(s)
    cache = steps.TokenCache(**{k: v for k, v in s.items() if k not in "KV"}, K=s["K"], V=s["V"], n_sink=n_sink, n_local=n_local)
    for i in range(4):
        kv = _randn((B, 2, Hkv, D), 50 + i, DT[dtype])  # strided new rows
        S.cache_insert(want, to_np(kv[:, 0]), to_np(kv[:, 1]), T, n_sink, n_local)
        cache.insert(kv[:, 0], kv[:, 1])
        csa.csa_check_device_status()
        _same(s, want)
    assert not cache.counters.any()


def test_cache_insert_inactive_budget_and_bad_state(steps, csa):
    """Inactive sequences and slots behind the budget stay as they are; bad
    lengths and positions are reported, their sequence left alone, the others served."""
    B, Hkv, T, D = 5, 2, 40, 64
    s = _cache_state(B, Hkv, T, D, torch.bfloat16, 9)
    s["K"] = s["K"].transpose(1, 2).contiguous().transpose(1, 2)  # token-major storage
    s["lengths"][:] = 32
    s["next_pos"][1] = -1
    want = _host(s)
    cache = steps.TokenCache(s["K"], s["V"], budget=32, n_sink=1, n_local=4,
                             **{k: s[k] for k in ("lengths", "next_pos", "positions", "weights")})
    k, v = _randn((B, Hkv, D), 1, torch.bfloat16), _randn((B, Hkv, D), 2, torch.bfloat16)
    cache.insert(k, v)
    csa.csa_check_device_status()
    S.cache_insert(want, to_np(k), to_np(v), 32, 1, 4)
    _same(s, want)
    # sequence 2 claims more slots than the budget, all of 3's are sinks
    s["lengths"][2] = 33
    s["positions"][3] = 0
    want = _host(s)
    active = {b: want["next_pos"][b] for b in range(B)}
    cache.insert(k, v)
    with pytest.raises(csa.CsaError) as e:
        csa.csa_check_device_status()
    assert e.value.status == 5
    want["next_pos"][2] = -1
    want["next_pos"][3] = -1
    S.cache_insert(want, to_np(k), to_np(v), 32, 1, 4)
    want["next_pos"][2] = active[2]
    want["next_pos"][3] = active[3] + 1
    _same(s, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,Sn,T,D,n_sink,n_local,ties", [
    (1, 1, 1, 1, 64, 0, 0, False), (3, 2, 100, 33, 64, 4, 8, True), (2, 1, 4097, 1000, 128, 4, 100, True),
    (1, 2, 20000, 513, 64, 0, 0, True), (4, 3, 700, 700, 80, 1, 1, False), (1, 8, 40000, 256, 64, 4, 252, False),
    (20, 8, 9000, 31, 6, 2, 3, True)])
def test_cache_compress(steps, csa, dtype, B, Hkv, Sn, T, D, n_sink, n_local, ties):
    src = _cache_state(B, Hkv, Sn, D, DT[dtype], Sn + T, True, ties)
    rng = np.random.default_rng(Sn)
    n = rng.integers(0, Sn + 1, B)
    n[0] = Sn
    n[-1] = min(n[-1], T) if B > 2 else n[-1]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    K = src["K"].transpose(1, 2).contiguous().transpose(1, 2)  # token-major storage
    for given in (False, True):
        dst = _cache_state(B, Hkv, T, D, DT[dtype], 3, True)
        want = _host(dst)
        cache = steps.TokenCache(**{k: v for k, v in dst.items() if k not in "KV"}, K=dst["K"], V=dst["V"],
                                 n_sink=n_sink, n_local=n_local)
        kw = dict(positions=src["positions"], next_pos=src["next_pos"]) if given else {}
        cache.compress(K, src["V"], src["weights"], lengths=lens, **kw)
        csa.csa_check_device_status()
        h = _host(src)
        kept = S.cache_compress(h["weights"], n, T, n_sink, n_local, *((h["positions"], h["next_pos"]) if given else ()))
        for b in range(B):
            want["lengths"][b] = min(n[b], T)
            want["next_pos"][b] = h["next_pos"][b] if given else n[b]
            for u in range(Hkv):
                rows = kept[b][u]
                m = len(rows)
                for name in ("K", "V", "weights"):
                    want[name][b, u, :m] = h[name][b, u, rows]
                want["positions"][b, u, :m] = h["positions"][b, u, rows] if given else rows
        _same(dst, want)


@pytest.mark.parametrize("B,Hkv,Sn,T,ties", [(1, 1, 65541, 65541, True), (2, 2, 70001, 300, True), (1, 3, 131072, 40000, False),
                                              (4, 8, 40003, 100, True), (9, 8, 20001, 77, True), (10, 8, 9001, 50, False)])
def test_cache_compress_many_rows(steps, csa, B, Hkv, Sn, T, ties):
    """Many rows a unit: CTAs, alone and in clusters of two, four and eight, with
    more threads each."""
    test_cache_compress(steps, csa, "bf16", B, Hkv, Sn, T, 8, 4, 10, ties)


def test_cache_compress_keys_beyond_shared_memory(steps, csa):
    """More rows than eight CTAs hold keys for: they are read again each pass."""
    Sn, T = 8 * 49152 + 5, 64
    w = torch.rand(1, 1, Sn, device="cuda")
    K = torch.arange(Sn, device="cuda", dtype=torch.float32).view(1, 1, Sn, 1).expand(1, 1, Sn, 4).contiguous()
    cache = steps.TokenCache(torch.zeros(1, 1, T, 4, device="cuda"), torch.zeros(1, 1, T, 4, device="cuda"), n_sink=2, n_local=2)
    cache.compress(K, K, w)
    csa.csa_check_device_status()
    kept = S.cache_compress(to_np(w), [Sn], T, 2, 2)[0][0]
    assert cache.positions[0, 0].tolist() == kept and cache.K[0, 0, :, 3].tolist() == kept


def test_cache_refuses(csa, steps):
    K = torch.zeros(1, 2, 64, 64, device="cuda")
    w = torch.zeros(1, 2, 64, device="cuda")
    cache = steps.TokenCache(K, torch.zeros_like(K), budget=32)
    with pytest.raises(csa.CsaError):
        cache.compress(K, torch.zeros_like(K), w)  # source and cache overlap
    with pytest.raises(csa.CsaError):
        cache.compress(torch.zeros_like(K), torch.zeros_like(K), w, lengths=cache.lengths)
    with pytest.raises(csa.CsaError):
        cache.insert(K[:, :, 0].half(), K[:, :, 0])
    with pytest.raises(csa.CsaError):
        steps.TokenCache(K, torch.zeros_like(K), n_sink=60, n_local=4).insert(K[:, :, 0], K[:, :, 0])
    with pytest.raises(csa.CsaError):  # one slot's storage for all
        steps.TokenCache(K[:, :, :1].expand(1, 2, 64, 64), torch.zeros_like(K)).insert(K[:, :, 0], K[:, :, 0])


# ---------------------------------------------------------------- decode

def _decode_case(dtype, B, Hkv, G, D, N, Tp, T, plens, starts, lens, seed, token_major=False, poison=True):
    Hq = Hkv * G
    q = _randn((B, Hq, D), seed, DT[dtype])
    K, V = _randn((B, Hkv, T, D), seed + 1, DT[dtype]), _randn((B, Hkv, T, D), seed + 2, DT[dtype])
    Kp, Vp = _randn((N, Hkv, Tp, D), seed + 3, DT[dtype]), _randn((N, Hkv, Tp, D), seed + 4, DT[dtype])
    if poison:  # what lies behind the lengths must not matter
        for b in range(B):
            K[b, :, lens[b]:], V[b, :, lens[b]:] = float("nan"), float("inf")
        for n in range(N):
            Kp[n, :, plens[n]:], Vp[n, :, plens[n]:] = float("inf"), float("nan")
    if token_major:
        K, V, Kp, Vp = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (K, V, Kp, Vp))
    return q, K, V, Kp, Vp


def _decode_check(steps, csa, dtype, B, Hkv, G, D, N, Tp, T, plens, starts, lens, seed=1, out_dtype=torch.float32,
                  decay=1.0, accumulate=True, scale=None, **kw):
    q, K, V, Kp, Vp = _decode_case(dtype, B, Hkv, G, D, N, Tp, T, plens, starts, lens, seed, **kw)
    w0 = _randn((B, Hkv, T), seed + 9).abs()
    if decay == 0.0:
        w0[:] = float("nan")  # not read
    cache = steps.TokenCache(K, V, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), weights=w0.clone())
    pk = {}
    if N:
        pk = dict(Kp=Kp, Vp=Vp, prefix_len=torch.tensor(plens, dtype=torch.int32, device="cuda"),
                  group_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, accumulate=accumulate, decay=decay, scale=scale, out_dtype=out_dtype, **pk)
    dec.workspace.fill_(255)  # NaNs: nothing of it may be taken for a value
    out, lse = dec.attend(q)
    csa.csa_check_device_status()
    scale = 1 / math.sqrt(D) if scale is None else scale
    a = [to_np(x) for x in (q, K, V)]
    p = [to_np(Kp), to_np(Vp), plens, starts] if N else [None] * 4
    ro, rl, rw, spread = S.prefix_decode(a[0], a[1], a[2], lens, scale, *p, weights=to_np(w0), decay=decay)
    # E: the largest absolute sum of a logit, in roundings
    big = 0.0
    for b in range(B):
        for keys in [a[1][b, :, :lens[b]]] + ([p[0][n, :, :plens[n]] for n in range(N) if starts[n] <= b < starts[n + 1]]):
            if keys.size:
                qa = np.abs(a[0][b]).reshape(Hkv, G, D)
                big = max(big, float(np.einsum("hgd,htd->hgt", qa, np.abs(keys)).max()) * scale)
    E = (D + 4) * U32 * big
    rel = 2 * E + 2.0 ** -20
    got = to_np(out)
    u = U16 if out_dtype == torch.bfloat16 else U32
    tol = u * np.abs(ro) + (rel + (U16 if dtype == "bf16" else 0.0)) * spread * (1 + u) + 1e-30
    assert int(np.isfinite(got).sum()) == got.size
    assert np.all(np.abs(got - ro) <= tol), (np.abs(got - ro) / tol).max()
    gl = to_np(lse)
    assert np.array_equal(np.isinf(gl), np.isinf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(gl[fin] - rl[fin]) <= E + 2.0 ** -20 + 4 * U32 * np.abs(rl[fin]))
    gw = to_np(cache.weights)
    if not accumulate:
        assert np.array_equal(gw, to_np(w0))
        return
    for b in range(B):
        n = lens[b]
        assert np.array_equal(gw[b, :, n:], to_np(w0)[b, :, n:], equal_nan=True)  # behind the length: as it was
        old = decay * to_np(w0)[b, :, :n] if decay else 0.0
        new = rw[b, :, :n] - old
        assert np.all(np.abs(gw[b, :, :n] - rw[b, :, :n]) <= rel * new + 8 * U32 * rw[b, :, :n] + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 16])
def test_decode_group_sizes(steps, csa, dtype, D, G):
    _decode_check(steps, csa, dtype, 5, 2, G, D, 1, 200, 130, [173], [0, 5], [0, 1, 64, 65, 130])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [1, 15, 63, 64, 65, 127, 128, 1000, 5003])
def test_decode_lengths(steps, csa, dtype, P):
    _decode_check(steps, csa, dtype, 3, 2, 4, 128, 1, P + 7, max(P, 2), [P], [0, 3], [P, 0, max(1, P // 2)], seed=P)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,G,D,N,Tp,T,plens,starts,lens", [
    (6, 2, 4, 128, 3, 300, 70, [300, 0, 129], [0, 2, 3, 6], [70, 0, 5, 64, 1, 33]),   # an empty prefix
    (6, 1, 4, 64, 2, 257, 9, [257, 31], [1, 1, 4], [0, 9, 0, 1, 0, 3]),               # an empty group, loose sequences
    (4, 2, 2, 128, 0, 0, 100, [], [], [100, 0, 1, 99]),                               # no prefix at all
    (3, 2, 4, 64, 1, 640, 1, [640], [0, 3], [0, 0, 0]),                               # nothing of one's own
    (40, 1, 8, 128, 1, 333, 20, [333], [0, 40], [i % 21 for i in range(40)]),          # 320 rows: tiles of rows
    (33, 2, 4, 64, 1, 500, 64, [500], [0, 33], [64] * 33),                             # 132 rows
    (70, 1, 5, 128, 2, 200, 3, [200, 77], [3, 60, 70], [i % 4 for i in range(70)]),    # heads across tile borders
    (2, 1, 1, 64, 1, 70000, 4, [69999], [0, 2], [4, 2]),                               # long: every SM on one unit
])
def test_decode_groups(steps, csa, dtype, B, Hkv, G, D, N, Tp, T, plens, starts, lens):
    _decode_check(steps, csa, dtype, B, Hkv, G, D, N, Tp, T, plens, starts, lens, seed=B + Tp)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out_dtype,decay,accumulate,token_major", [
    (torch.bfloat16, 1.0, True, True), (torch.float32, 0.0, True, False), (torch.bfloat16, 0.5, True, False),
    (torch.float32, 1.0, False, True)])
def test_decode_options(steps, csa, dtype, out_dtype, decay, accumulate, token_major):
    _decode_check(steps, csa, dtype, 4, 3, 4, 128, 2, 190, 150, [190, 100], [0, 1, 4], [150, 3, 0, 88], seed=77,
                  out_dtype=out_dtype, decay=decay, accumulate=accumulate, token_major=token_major, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_sharp_softmax(steps, csa, dtype):
    """Large scales: the running maximum moves by hundreds between chunks."""
    _decode_check(steps, csa, dtype, 3, 1, 4, 64, 1, 900, 200, [900], [0, 2], [200, 7, 130], seed=5, scale=6.0)


def test_decode_bad_lengths_are_reported(steps, csa):
    """Lengths and group bounds out of range are clamped and reported."""
    B, Hkv, G, D, T, Tp = 3, 1, 4, 64, 64, 100
    q, K, V, Kp, Vp = _decode_case("bf16", B, Hkv, G, D, 2, Tp, T, [100, 50], [0, 2, 3], [64, 10, 5], 3, poison=False)

    def run(lens, plens, starts):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        cache = steps.TokenCache(K, V, lengths=i32(lens))
        dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=Kp, Vp=Vp, prefix_len=i32(plens), group_start=i32(starts))
        out, lse = dec.attend(q)
        return out.clone(), lse.clone()

    for bad, good in [(([65, -3, 5], [100, 50], [0, 2, 3]), ([64, 0, 5], [100, 50], [0, 2, 3])),
                      (([64, 10, 5], [101, -1], [0, 2, 3]), ([64, 10, 5], [100, 0], [0, 2, 3])),
                      (([64, 10, 5], [100, 50], [-1, 2, 9]), ([64, 10, 5], [100, 50], [0, 2, 3])),
                      (([64, 10, 5], [100, 50], [2, 0, 3]), ([64, 10, 5], [100, 50], [2, 2, 3]))]:
        got = run(*bad)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_check_device_status()
        assert e.value.status == 5
        want = run(*good)
        csa.csa_check_device_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_refuses(csa, steps):
    K = torch.zeros(2, 2, 64, 128, device="cuda", dtype=torch.bfloat16)
    cache = steps.TokenCache(K, torch.zeros_like(K))
    q = torch.zeros(2, 8, 128, device="cuda", dtype=torch.bfloat16)
    dec = steps.SharedPrefixDecoder(cache, Hq=8)
    with pytest.raises(csa.CsaError):
        dec.attend(q.float())
    with pytest.raises(csa.CsaError):
        dec.attend(q[:, ::2])
    dec.desc.workspace_bytes -= 1
    with pytest.raises(csa.CsaError):
        dec.attend(q)
    with pytest.raises(csa.CsaError):
        steps.SharedPrefixDecoder(cache, Hq=8, Kp=K, Vp=K).attend(q)  # two prefixes, no groups
    with pytest.raises(csa.CsaError):
        steps.SharedPrefixDecoder(cache, Hq=8, Kp=K.float(), Vp=K)
    odd = torch.zeros(2, 2, 64, 129, device="cuda", dtype=torch.bfloat16)[..., :128]
    with pytest.raises(csa.CsaError):  # rows that start off 16 bytes
        steps.SharedPrefixDecoder(steps.TokenCache(odd, odd), Hq=8).attend(q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_steps_back_to_back(steps, dtype):
    """Steps in a row, with and without waiting between them: a step's merge
    reads the sums ahead of its attention, but not ahead of the step before."""
    B, Hkv, G, D, T, Tp = 7, 2, 4, 64, 90, 700
    q, K, V, Kp, Vp = _decode_case(dtype, B, Hkv, G, D, 1, Tp, T, [Tp], [0, 5], [T] * B, 8, poison=False)
    k, v = K[:, :, 0].contiguous(), V[:, :, 1].contiguous()
    outs = []
    for wait in (True, False):
        cache = steps.TokenCache(K.clone(), V.clone(), lengths=torch.full((B,), T - 3, dtype=torch.int32, device="cuda"),
                                 next_pos=torch.full((B,), T - 3, dtype=torch.int32, device="cuda"), budget=T - 1)
        dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=Kp, Vp=Vp, decay=0.9,
                                        group_start=torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
        for _ in range(60):
            out, lse = dec.step(q, k, v)
            if wait:
                torch.cuda.synchronize()
        outs.append((out.clone(), lse.clone(), cache.weights.clone(), cache.positions.clone(), cache.K.clone()))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_decode_is_deterministic(steps):
    """No sum depends on the order in which SMs finish."""
    q, K, V, Kp, Vp = _decode_case("bf16", 9, 2, 4, 128, 1, 3000, 300, [3000], [0, 9], [300] * 9, 4, poison=False)
    outs = []
    for _ in range(3):
        cache = steps.TokenCache(K, V, lengths=torch.full((9,), 300, dtype=torch.int32, device="cuda"))
        dec = steps.SharedPrefixDecoder(cache, Hq=8, Kp=Kp, Vp=Vp)
        out, lse = dec.attend(q)
        outs.append((out.clone(), lse.clone(), cache.weights.clone()))
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_steps(steps, csa, dtype):
    """Prompts compressed into caches, then decode steps that turn, insert over
    the lightest token and attend: eager first, then the same step captured and
    replayed, against the oracle step by step."""
    B, Hkv, G, D, T, Tp, Sn = 4, 2, 4, 64, 40, 150, 90
    n_sink, n_local = 2, 6
    dt = DT[dtype]
    Kp, Vp = _randn((1, Hkv, Tp, D), 1, dt), _randn((1, Hkv, Tp, D), 2, dt)
    Ks, Vs = _randn((B, Hkv, Sn, D), 3, dt), _randn((B, Hkv, Sn, D), 4, dt)
    ws = torch.rand(B, Hkv, Sn, device="cuda")
    plen = [90, 12, 40, 0]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = steps.TokenCache(*(torch.zeros(B, Hkv, T, D, dtype=dt, device="cuda") for _ in range(2)), n_sink=n_sink, n_local=n_local)
    cache.compress(Ks, Vs, ws, lengths=i32(plen))
    rot = steps.Rotary(32, theta=10000.0, scaling="turns", factor=4.0, orig_len=64)
    w = S.rotary_freqs(32, 10000.0, "turns", 4.0, 64)
    dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=Kp, Vp=Vp, group_start=i32([0, 3]), rotary=rot)
    state = dict(K=cache.K, V=cache.V, weights=cache.weights, positions=cache.positions, lengths=cache.lengths,
                 next_pos=cache.next_pos)
    q, k, v = (torch.zeros(B, n, D, dtype=dt, device="cuda") for n in (Hkv * G, Hkv, Hkv))

    def one():
        dec.step(q, k, v)

    graph = None
    for i in range(60):
        if i == 30:
            saved = {n: x.clone() for n, x in state.items()}
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                one()
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, capture_error_mode="relaxed"):
                one()
            for n, x in state.items():
                x.copy_(saved[n])
        for t, s in ((q, 10), (k, 11), (v, 12)):
            t.copy_(_randn(t.shape, 100 * i + s, dt))
        want = _host(state)  # the oracle takes each step from the GPU's state
        pos = want["next_pos"].copy()
        graph.replay() if graph else one()
        csa.csa_check_device_status()
        # the turned query and key are checked as such; the oracle goes on with them
        _rotary_close(dec.q[:, None], q[:, None], pos[:, None], w, "half", 1.0, False)
        _rotary_close(dec.k[:, None], k[:, None], pos[:, None], w, "half", 1.0, False)
        S.cache_insert(want, to_np(dec.k), to_np(v), T, n_sink, n_local)
        for n in ("K", "V", "positions", "lengths", "next_pos"):
            got = to_np(state[n]) if state[n].dtype.is_floating_point else state[n].cpu().numpy()
            assert np.array_equal(got, want[n]), (i, n)
        ro, rl, rw, spread = S.prefix_decode(to_np(dec.q), want["K"], want["V"], want["lengths"], 1 / math.sqrt(D),
                                             to_np(Kp), to_np(Vp), [Tp], [0, 3], want["weights"])
        # D = 64: E <= 68 u * sum |q k| / 8 < 68 * 2^-24 * 12 = 5e-5
        rel = 1e-4 + 2.0 ** -20
        tol = (rel + (U16 if dtype == "bf16" else 0)) * spread + U32 * np.abs(ro)
        assert np.all(np.abs(to_np(dec.out) - ro) <= tol), i
        assert np.all(np.abs(to_np(dec.lse) - rl) <= 5e-5 + 2.0 ** -20 + 4 * U32 * np.abs(rl))
        assert np.all(np.abs(to_np(cache.weights) - rw) <= rel * rw + 1e-30)
    assert cache.lengths.tolist() == [T] * B


def test_two_streams_with_their_own_workspaces(steps, csa):
    """Two decoders over one prefix run at once on two streams."""
    Kp, Vp = _randn((1, 2, 4000, 128), 1, torch.bfloat16), _randn((1, 2, 4000, 128), 2, torch.bfloat16)
    decs, qs = [], []
    for i in range(2):
        K, V = _randn((6, 2, 200, 128), 10 + i, torch.bfloat16), _randn((6, 2, 200, 128), 20 + i, torch.bfloat16)
        cache = steps.TokenCache(K, V, lengths=torch.full((6,), 200, dtype=torch.int32, device="cuda"))
        decs.append(steps.SharedPrefixDecoder(cache, Hq=8, Kp=Kp, Vp=Vp, decay=0.0))
        qs.append(_randn((6, 8, 128), 30 + i, torch.bfloat16))
    want = []
    for d, q in zip(decs, qs):
        d.attend(q)
        want.append((d.out.clone(), d.lse.clone(), d.cache.weights.clone()))
        d.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for d, q, s in zip(decs, qs, streams):
            d.attend(q, stream=s)
    torch.cuda.synchronize()
    csa.csa_check_device_status()
    for d, (o, l, w) in zip(decs, want):
        assert torch.equal(d.out, o) and torch.equal(d.lse, l) and torch.equal(d.cache.weights, w)


# ---------------------------------------------------------------- what no ordinary call has

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [4, 12])
def test_decode_nan_stays_in_its_rows(steps, csa, dtype, G):
    """A NaN or infinity in a query or in a valid key makes the rows that see it NaN,
    the others keep their values."""
    B, Hkv, D, T, Tp = 20, 2, 64, 150, 200
    lens = [150] * B
    q, K, V, Kp, Vp = _decode_case(dtype, B, Hkv, G, D, 1, Tp, T, [Tp], [0, 16], lens, 8, poison=False)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def run():
        cache = steps.TokenCache(K, V, lengths=i32(lens), weights=torch.zeros(B, Hkv, T, device="cuda"))
        dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=Kp, Vp=Vp, group_start=i32([0, 16]))
        out, lse = dec.attend(q)
        csa.csa_check_device_status()
        return out.clone(), lse.clone(), cache.weights.clone()

    want = run()
    q[3, G + 1, 5] = float("nan")           # one row
    K[17, 1, 77, 0] = float("nan")          # the rows of one sequence and KV head
    K[18, 0, 3] = float("inf")
    got = run()
    bad = torch.zeros(B, Hkv * G, dtype=torch.bool, device="cuda")
    bad[3, G + 1] = True
    bad[17, G:] = True
    # K = inf in all D: q.k is a sum of both infinities, or all of one sign by chance
    free = torch.ones(B, Hkv * G, dtype=torch.bool, device="cuda")
    free[18, :G] = False
    assert bool(torch.isnan(got[1][bad]).all()) and bool(torch.isnan(got[0][bad]).all())
    keep = ~bad & free
    assert torch.equal(got[1][keep], want[1][keep]) and torch.equal(got[0][keep], want[0][keep])
    assert bool(torch.isnan(got[2][17, 1]).all()) and torch.equal(got[2][17, 0], want[2][17, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_many_sequences(steps, csa, dtype):
    """More sequences than the threads of a block: the split takes several rounds."""
    B = 700
    lens = [(i * 37) % 34 for i in range(B)]
    _decode_check(steps, csa, dtype, B, 1, 2, 64, 3, 90, 33, [90, 0, 41], [0, 300, 301, 690], lens, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_broadcast_storage(steps, csa, dtype):
    """Keys and values stored once for all heads, or for all sequences."""
    B, Hkv, G, D, T, Tp = 3, 4, 4, 128, 90, 150
    dt = DT[dtype]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = _randn((B, Hkv * G, D), 1, dt)
    Kp, Vp = (_randn((1, 1, Tp, D), s, dt).expand(1, Hkv, Tp, D) for s in (2, 3))
    K, V = (_randn((1, Hkv, T, D), s, dt).expand(B, Hkv, T, D) for s in (4, 5))

    def run(*kv):
        cache = steps.TokenCache(kv[0], kv[1], lengths=i32([90, 17, 64]))
        dec = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=kv[2], Vp=kv[3])
        out, lse = dec.attend(q)
        csa.csa_check_device_status()
        return out.clone(), lse.clone(), cache.weights.clone()

    for x, y in zip(run(K, V, Kp, Vp), run(*(t.contiguous() for t in (K, V, Kp, Vp)))):
        assert torch.equal(x, y)


def test_offsets_beyond_32_bits(steps, csa):
    """Keys and values of more than 2^31 elements: prefix, own cache, insert and
    compress at their far ends."""
    H, T, D = 2, 8_500_000, 128
    K = torch.zeros(1, H, T, D, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    q = _randn((1, 8, D), 1, torch.bfloat16)
    spots = [0, T // 2 + 3, T - 1]
    for i, t in enumerate(spots):
        K[0, :, t] = (q[0, ::4] * (1 + 0.01 * i)).to(torch.bfloat16)
        V[0, :, t] = _randn((H, D), 20 + i, torch.bfloat16)
    # T keys of logit 0 (less the spots), and the spots
    qd = q[0].double().view(H, 4, D)
    logits = torch.stack([torch.einsum("hgd,hd->hg", qd, K[0, :, t].double()) / D ** 0.5 for t in spots], -1)
    for as_prefix in (False, True):
        if as_prefix:
            cache = steps.TokenCache(K[:, :, :1], V[:, :, :1])
            dec = steps.SharedPrefixDecoder(cache, Hq=8, Kp=K, Vp=V)
        else:
            cache = steps.TokenCache(K, V, lengths=torch.tensor([T], dtype=torch.int32, device="cuda"), n_local=4)
            dec = steps.SharedPrefixDecoder(cache, Hq=8)
        out, lse = dec.attend(q)
        csa.csa_check_device_status()
        want = torch.logsumexp(torch.cat([logits, torch.full((H, 4, 1), math.log(T - 3), device="cuda")], -1), -1)
        # a partial's sum takes at most 2^12 steps, each off by 2^-24 of it: 2.5e-4 of l, of a weight and of lse
        assert (lse[0].view(H, 4) - want).abs().max() < 1e-3
        p = (logits - want[..., None]).exp()
        ref = torch.einsum("hgs,hsd->hgd", p, torch.stack([V[0, :, t].double() for t in spots], 1))
        size = torch.einsum("hgs,hsd->hgd", p, torch.stack([V[0, :, t].double().abs() for t in spots], 1))
        assert bool(((out[0].view(H, 4, D).double() - ref).abs() <= (U16 + 4e-3) * size + 1e-6).all())
    assert (cache.weights.numel() == H)  # the prefix run's own cache; the first one's is below
    cache = steps.TokenCache(K, V, lengths=torch.tensor([T], dtype=torch.int32, device="cuda"),
                             next_pos=torch.tensor([T], dtype=torch.int32, device="cuda"), n_local=2)
    cache.positions.copy_(torch.arange(T, dtype=torch.int32, device="cuda").expand(1, H, T))
    cache.weights.fill_(1.0)
    cache.weights[0, :, T - 3] = 0.5
    k, v = _randn((1, H, D), 30, torch.bfloat16), _randn((1, H, D), 31, torch.bfloat16)
    cache.insert(k, v)
    csa.csa_check_device_status()
    assert torch.equal(K[0, :, T - 3], k[0]) and torch.equal(V[0, :, T - 3], v[0])
    assert cache.positions[0, :, T - 3].tolist() == [T, T]
    small = steps.TokenCache(*(torch.zeros(1, H, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)), n_sink=1, n_local=2)
    w = torch.rand(1, H, T, device="cuda")
    small.compress(K, V, w)
    csa.csa_check_device_status()
    for h in range(H):
        top = torch.sort(w[0, h, 1:T - 2], descending=True, stable=True)[1][:5] + 1
        rows = sorted([0, T - 2, T - 1] + top.tolist())
        assert small.positions[0, h].tolist() == rows
        assert torch.equal(small.K[0, h], K[0, h, rows]) and torch.equal(small.V[0, h], V[0, h, rows])


def test_rotary_offsets_beyond_32_bits(steps):
    S, H, D = 131072, 160, 128
    x = torch.zeros(1, S, H, D, dtype=torch.bfloat16, device="cuda")
    x[:, -3:] = _randn((1, 3, H, D), 4, torch.bfloat16)
    before = x[:, -3:].clone()
    steps.Rotary(128).rotate(x, q_out=x)
    _rotary_close(x[:, -3:], before, np.arange(S - 3, S)[None], oracle_freqs(128, 10000.0), "half", 1.0, False)
    assert not x[:, :-3].any()


def test_empty_batches(steps, csa):
    K = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = steps.TokenCache(K, K.clone())
    cache.insert(K[:, :, 0], K[:, :, 0])
    cache.compress(K, K.clone(), torch.zeros(0, 2, 16, device="cuda"))
    out, lse = steps.SharedPrefixDecoder(cache, Hq=4).attend(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    csa.csa_check_device_status()


def test_rotary_outputs_belong_to_the_stream(steps, csa):
    """Without outputs, a torch stream allocates them; a raw one needs them."""
    x = _randn((2, 5, 3, 64), 1)
    r = steps.Rotary(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = r.rotate(x, pos0=7, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, r.rotate(x, pos0=7))
    with pytest.raises(csa.CsaError):
        r.rotate(x, stream=side.cuda_stream)
    with pytest.raises(csa.CsaError):
        r.rotate(x.half())
    with pytest.raises(csa.CsaError):
        steps.TokenCache(x.half(), x.half())
