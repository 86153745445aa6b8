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
    cache = steps.TokenCache(K, K.clone(), lengths=_i32([40, 3, 0]), next_pos=_i32([0, -1, -2, -(1 << 31)])[1:],
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


# ---------------------------------------------------------------- gradients of the rotation

def _tol(x, amp):
    """Of a turned tensor: 6e-7 A (|x_a| + |x_b|) and the result's rounding (the bound of the
    forward tests), over all its values."""
    u = U16 if x.dtype == torch.bfloat16 else U32
    return float((2 * 6e-7 + u * math.sqrt(2)) * amp * x.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("what", ["both", "q", "k", "no k", "unused k", "expanded"])
def test_rotary_autograd(steps, dtype, layout, what):
    """Gradients flow through rotate() as the formula says, from packed projections, for
    positions that change after the forward pass."""
    B, Sq, Hq, Hkv, D, rot, amp = 2, 33, 6, 2, 64, 48, 1.25
    packed = _randn((B, Sq, (Hq + 2 * Hkv) * D), 7, DT[dtype])
    need = {"q": (True, False), "k": (False, True)}.get(what, (True, True))
    q0 = packed[..., :Hq * D].view(B, Sq, Hq, D).clone().requires_grad_(need[0])
    k0 = packed[..., Hq * D:(Hq + Hkv) * D].view(B, Sq, Hkv, D).clone().requires_grad_(need[1])
    q, k = q0.transpose(1, 2).contiguous().transpose(1, 2), k0 * 1  # head-major, and a plain copy
    pos = np.random.default_rng(3).integers(0, 1 << 20, (B, Sq))
    p = _i32(pos.tolist())
    r = steps.Rotary(rot, layout=layout, amplitude=amp)
    w = S.rotary_freqs(rot, 10000.0)
    with torch.no_grad():
        plain = r.rotate(q, positions=p) if what == "no k" else r.rotate(q, k, positions=p)
    y = r.rotate(q, None if what == "no k" else k, positions=p)
    yq, yk = (y, None) if what == "no k" else y
    assert torch.equal(yq, plain if what == "no k" else plain[0])
    assert yq.requires_grad and (yk is None or yk.requires_grad)
    p.zero_()  # the gradient is that of the positions that were turned by
    gq, gk = _randn((B, Sq, Hq, D), 8, DT[dtype]), _randn((B, Sq, Hkv, D), 9, DT[dtype])
    if what == "expanded":
        gq, gk = torch.ones_like(gq), torch.ones_like(gk)
        loss = yq.sum() + yk.sum()
    else:
        loss = (yq * gq).sum() + (0 if yk is None or what == "unused k" else (yk * gk).sum())
    loss.backward()
    for x, g, used in ((q0, gq, need[0]), (k0, gk, need[1] and what not in ("no k", "unused k"))):
        if not used:
            assert x.grad is None or not x.grad.any()
            continue
        want = S.rotary(to_np(g), pos, w, layout, amp, transpose=True)
        want[..., rot:] = to_np(g)[..., rot:]
        assert np.abs(to_np(x.grad) - want).max() <= _tol(g, amp)


def test_rotary_autograd_against_differences(steps):
    """Central differences of a linear map are exact up to rounding, and the gradient is
    itself differentiable."""
    B, Sq, H, D, amp = 1, 3, 2, 8, 0.75
    r = steps.Rotary(6, theta=100.0, layout="interleaved", amplitude=amp)
    x, c = _randn((B, Sq, H, D), 1).requires_grad_(), _randn((B, Sq, H, D), 2).requires_grad_()
    f = lambda x, c: (r.rotate(x, pos0=11) * c).sum()
    g, = torch.autograd.grad(f(x, c), x, create_graph=True)
    num = torch.zeros_like(x)
    with torch.no_grad():
        for i in np.ndindex(*x.shape):
            e = torch.zeros_like(x)
            e[i] = 1.0
            num[i] = ((r.rotate(x + e, pos0=11) - r.rotate(x - e, pos0=11)).double() * c.double()).sum() / 2
    # each difference: two roundings of values below 8 and the rotation's 6e-7 of |x| sums, times c
    assert float((g.detach() - num).abs().max()) <= 8 * (U32 + 2 * 6e-7) * float(c.detach().abs().max()) * 2
    v = _randn(x.shape, 3)
    h, = torch.autograd.grad((g * v).sum(), c)  # d/dc of c . rotate(v)
    with torch.no_grad():
        assert torch.equal(h, r.rotate(v, pos0=11))


@pytest.mark.parametrize("pad", [(1, 1), (1, 2), (2, 2), (0, 3)])
def test_rotary_autograd_of_a_narrow_gradient(steps, pad):
    """The gradient comes back as a view of a wider one, off the pairs' alignment."""
    x = _randn((2, 5, 3, 64), 1, torch.bfloat16).requires_grad_()
    c = _randn((2, 5, 3, 64 + sum(pad)), 2, torch.bfloat16)
    r = steps.Rotary(64, layout="interleaved")
    parts = [torch.zeros(2, 5, 3, n, dtype=x.dtype, device="cuda") for n in pad]
    (torch.cat([parts[0], r.rotate(x, pos0=3), parts[1]], -1) * c).sum().backward()
    with torch.no_grad():
        want = r.rotate(c[..., pad[0]:pad[0] + 64].contiguous(), pos0=3, transpose=True)
    assert torch.equal(x.grad, want)


def test_rotary_autograd_in_a_graph(steps):
    """A captured training step gives the eager one's gradients on new inputs."""
    r = steps.Rotary(64, theta=10000.0)
    x, g = _randn((2, 17, 4, 64), 1), _randn((2, 17, 4, 64), 2)
    k, gk = _randn((2, 17, 1, 64), 3), _randn((2, 17, 1, 64), 4)
    p = torch.arange(17, dtype=torch.int32, device="cuda").expand(2, 17)

    def step():
        xi, ki = x.detach().requires_grad_(), k.detach().requires_grad_()
        y, z = r.rotate(xi, ki, positions=p)
        return torch.autograd.grad([y, z], [xi, ki], [g, gk])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        out = step()
    g.copy_(_randn(g.shape, 5))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_rotary_refuses_what_autograd_cannot_see(steps, csa):
    r = steps.Rotary(64)
    x = _randn((1, 4, 2, 64), 1).requires_grad_()
    for kw in (dict(q_out=torch.empty_like(x)), dict(stream=torch.cuda.Stream())):
        with pytest.raises(csa.CsaError):
            r.rotate(x, **kw)
    with pytest.raises(csa.CsaError):
        r.rotate(x.detach(), x, k_out=torch.empty_like(x))
    with torch.no_grad():
        y = torch.empty_like(x)
        assert r.rotate(x, q_out=y) is y and not y.requires_grad


def test_step_takes_outputs_of_a_model_in_training_mode(steps, csa):
    K = _randn((2, 2, 16, 64), 1)
    cache = steps.TokenCache(K, K.clone())
    dec = steps.SharedPrefixDecoder(cache, Hq=4, rotary=steps.Rotary(64))
    q, k, v = (_randn((2, n, 64), n).requires_grad_() for n in (4, 2, 2))
    out, _ = dec.step(q, k, v)
    csa.csa_check_device_status()
    assert not out.requires_grad and torch.equal(out.view(2, 2, 2, 64), v.detach()[:, :, None].expand(2, 2, 2, 64))


# ---------------------------------------------------------------- strides that are not used

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_odd_strides_of_single_entries(steps, csa, dtype):
    """One prefix, one sequence, one token or one head out of wider buffers: the same bits
    as from dense ones."""
    dt = DT[dtype]

    def odd(shape, seed):
        """A tensor whose one-entry indices have strides that no row could start on."""
        dense = _randn(shape, seed, dt)
        st = [s if n > 1 else 3 + 2 * i for i, (n, s) in enumerate(zip(shape, dense.stride()))]
        return dense, dense.as_strided(shape, st)

    B, Hkv, T, Tp, D = 1, 1, 50, 200, 128
    for G in (4, 12):
        pairs = [odd(s, i) for i, s in enumerate([(B, Hkv, T, D), (B, Hkv, T, D), (1, Hkv, Tp, D), (1, Hkv, Tp, D)])]
        q = _randn((B, Hkv * G, D), 9, dt)
        got = []
        for way in (0, 1):
            K, V, Kp, Vp = (p[way] for p in pairs)
            cache = steps.TokenCache(K, V, lengths=_i32([T]))
            out, lse = steps.SharedPrefixDecoder(cache, Hq=Hkv * G, Kp=Kp, Vp=Vp).attend(q)
            csa.csa_check_device_status()
            got.append((out.clone(), lse.clone(), cache.weights.clone()))
        assert all(torch.equal(x, y) for x, y in zip(*got))
    r = steps.Rotary(64, layout="interleaved")
    for shape in ((1, 1, 3, 64), (1, 7, 1, 64), (2, 1, 1, 64), (1, 1, 1, 64)):
        dense, view = odd(shape, 3)
        want = r.rotate(dense, pos0=5, q_out=torch.empty_like(dense))
        assert torch.equal(r.rotate(view, pos0=5, q_out=torch.empty_like(dense)), want)
        assert torch.equal(r.rotate(view, pos0=5, q_out=view), want) and torch.equal(dense, want)
    (K, Kv), (V, Vv) = odd((1, 1, 8, 6), 1), odd((1, 1, 8, 6), 2)
    (k, kv), (v, vv) = odd((1, 1, 6), 3), odd((1, 1, 6), 4)
    cache = steps.TokenCache(Kv, Vv)
    cache.insert(kv, vv)
    csa.csa_check_device_status()
    assert torch.equal(K[0, 0, 0], k[0, 0]) and torch.equal(V[0, 0, 0], v[0, 0])


# ---------------------------------------------------------------- refused steps

@pytest.mark.parametrize("turned", [False, True])
def test_a_refused_step_leaves_the_cache_as_it_was(steps, csa, turned):
    K = _randn((2, 2, 16, 64), 1, torch.bfloat16)
    cache = steps.TokenCache(K, K.clone())
    q, k, v = (_randn((2, n, 64), n, torch.bfloat16) for n in (4, 2, 2))
    dec = steps.SharedPrefixDecoder(cache, Hq=4, rotary=steps.Rotary(64) if turned else None)
    before = {n: getattr(cache, n).clone() for n in ("K", "V", "weights", "positions", "lengths", "next_pos")}
    off = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4, 64)
    bad = [(q.float(), k, v), (q[:, :3], k, v), (q, k.float(), v), (q, k, v[:1]), (q, k[:, :1], v), (q.cpu(), k, v)]
    if not turned:  # (turned, the queries are copied)
        bad += [(off, k, v), (q.transpose(0, 1).contiguous().transpose(0, 1), k, v)]
    for args in bad:
        with pytest.raises(csa.CsaError):
            dec.step(*args)
        torch.cuda.synchronize()
        for n, x in before.items():
            assert torch.equal(getattr(cache, n), x), n
    dec.step(q, k, v)
    assert cache.lengths.tolist() == [1, 1]


def test_decoder_refuses_at_its_making(steps, csa):
    """What no call of it could do."""
    K = torch.zeros(2, 2, 64, 128, device="cuda", dtype=torch.bfloat16)
    cache = steps.TokenCache(K, torch.zeros_like(K))
    odd = torch.zeros(2, 2, 64, 129, device="cuda", dtype=torch.bfloat16)[..., :128]
    for kw in (dict(Kp=K, Vp=K), dict(scale=0.0), dict(scale=math.inf), dict(decay=-0.5), dict(decay=math.nan),
               dict(Kp=odd[:1], Vp=K[:1]), dict(Kp=K[:1], Vp=K[:1, :, :1].expand(1, 2, 64, 128))):
        with pytest.raises(csa.CsaError):
            steps.SharedPrefixDecoder(cache, Hq=8, **kw)
    with pytest.raises(csa.CsaError):
        steps.SharedPrefixDecoder(steps.TokenCache(odd, odd), Hq=8)


# ---------------------------------------------------------------- the last positions

def test_insert_at_the_last_positions(steps, csa):
    """2^31 - 2 is the last position that a token can take; at 2^31 - 1 the sequence is reported
    and left alone, and does not turn into an inactive one."""
    B, Hkv, T, D = 3, 2, 8, 64
    K = _randn((B, Hkv, T, D), 1)
    last = (1 << 31) - 2
    cache = steps.TokenCache(K, K.clone(), lengths=_i32([T, 3, T]), next_pos=_i32([last, last + 1, 20]), n_local=2,
                             positions=(torch.arange(T, dtype=torch.int32, device="cuda") + 5).expand(B, Hkv, T).contiguous())
    k, v = _randn((B, Hkv, D), 2), _randn((B, Hkv, D), 3)
    before = {n: getattr(cache, n).clone() for n in ("K", "V", "weights", "positions")}
    cache.insert(k, v)
    with pytest.raises(csa.CsaError) as e:
        csa.csa_check_device_status()
    assert e.value.status == 5
    assert cache.next_pos.tolist() == [last + 1, last + 1, 21] and cache.lengths.tolist() == [T, 3, T]
    for n, x in before.items():
        assert torch.equal(getattr(cache, n)[1], x[1])
    for b, at in ((0, last), (2, 20)):  # the lightest, the lowest of equals: slot 0
        assert cache.positions[b, :, 0].tolist() == [at] * Hkv and torch.equal(cache.K[b, :, 0], k[b])
    cache.insert(k, v)
    with pytest.raises(csa.CsaError):
        csa.csa_check_device_status()
    assert cache.next_pos.tolist() == [last + 1, last + 1, 22]
    assert not cache.counters.any()


# ---------------------------------------------------------------- the frequency table

def _two_pi():
    """2 pi to 60 digits, by Machin's formula."""
    from decimal import Decimal, getcontext
    getcontext().prec = 70

    def arctan_inv(n):
        total, term, k = Decimal(0), Decimal(1) / n, 0
        while abs(term) > Decimal(10) ** -68:
            total += term / (2 * k + 1) * (-1) ** k
            term, k = term / (n * n), k + 1
        return total
    return 8 * (4 * arctan_inv(5) - arctan_inv(239))


def _table(r):
    return [x % (1 << 64) for x in r.table.tolist()]


def _turns_off(table, exact):
    """Distance of a table's entries from exact turns per position, modulo one."""
    from decimal import Decimal
    off = []
    for got, t in zip(table, exact):
        d = (Decimal(got) / (1 << 64) - t) % 1
        off.append(float(min(abs(d), abs(1 - abs(d)))))
    return off


@pytest.mark.parametrize("rot,theta", [(128, 10000.0), (128, 500000.0), (64, 1000000.0), (2, 10000.0), (512, 1e8)])
def test_rotary_table_is_good_to_64_bit_floats(steps, rot, theta):
    """w = theta^(-2i/rot) in 64-bit floats: the exponent's rounding is |ln w| 2^-53 of
    w, pow at most two steps of 2^-52, 2 pi, the division and the exponent's own products 2^-53
    each: (|ln w| + 8) 2^-53 of w / 2 pi, and 2^-64 of the entry's last place."""
    from decimal import Decimal
    tau = _two_pi()
    r = steps.Rotary(rot, theta=theta)
    w = [Decimal(theta) ** (Decimal(-2 * i) / rot) for i in range(rot // 2)]
    off = _turns_off(_table(r), [x / tau for x in w])
    for i, (x, d) in enumerate(zip(w, off)):
        assert d <= (abs(math.log(float(x))) + 8) * 2.0 ** -53 * float(x / tau) + 2.0 ** -64, i
    print("largest error in turns at position 2^31: 2^%.1f" % math.log2(max(off) * 2.0 ** 31))


def test_rotary_table_of_own_frequencies(steps):
    """2 pi and the division, 2^-53 each of the whole number of turns; a negative frequency's
    turns are taken from one, 2^-54."""
    from decimal import Decimal
    tau = _two_pi()
    w = torch.cat([torch.rand(100, dtype=torch.float64) * 20 - 10, torch.rand(28, dtype=torch.float64) * 1e-6,
                   torch.tensor([-1e-9, 0.0, 6.0, -6.5], dtype=torch.float64)])
    r = steps.Rotary(2 * len(w), freqs=w.cuda())
    exact = [Decimal(x) / tau for x in w.tolist()]
    for x, d in zip(exact, _turns_off(_table(r), exact)):
        assert d <= 2 * 2.0 ** -53 * abs(float(x)) + (2.0 ** -54 if x < 0 else 0.0) + 2.0 ** -64


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_angles_wrap_exactly(steps, layout):
    """Position times table entry modulo a turn is exact: the result is that of the
    table's own frequency, at any 32-bit position."""
    rot = 128
    r = steps.Rotary(rot, theta=500000.0, layout=layout)
    pos = [0, 1, 131071, (1 << 31) - 1, (1 << 31) - 2, 1431655765, -1, -(1 << 31)]
    x = _randn((1, len(pos), 1, rot), 5)
    y = to_np(r.rotate(x, positions=_i32([pos])))[0, :, 0]
    xs = to_np(x)[0, :, 0]
    t = np.array([[(p * e) % (1 << 64) / 2.0 ** 64 for e in _table(r)] for p in pos]) * 2 * math.pi
    a, b = (xs[:, :64], xs[:, 64:]) if layout == "half" else (xs[:, ::2], xs[:, 1::2])
    u, v = a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)
    got = (y[:, :64], y[:, 64:]) if layout == "half" else (y[:, ::2], y[:, 1::2])
    for g, want in zip(got, (u, v)):
        assert np.all(np.abs(g - want) <= 6e-7 * (np.abs(a) + np.abs(b)) + U32 * np.abs(want))
