"""The serving operators around a bounded KV cache, as measured workloads.

Four operators, each in its plain form (elementary torch operations in 32 bits,
angles in 64) and through this package's own calls:

  rotary    rotary positions of the queries and keys (half or interleaved
            pairs, part of the head, scaled frequencies, or the gradient)
  decode    one query token per sequence over a prefix that several sequences
            share and over each sequence's own cache, with the weight that
            each own token received added to its running sum
  insert    a new token into a full cache, over the token of least weight
  compress  a prompt's tokens into a smaller cache, the heaviest kept
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def rotary_case(name, **kw):
    c = dict(name=name, op="rotary", dtype="bf16", B=1, S=1, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             theta=10000.0, scaling="none", factor=1.0, orig=8192, amplitude=1.0, far=131072, packed=False, gradient=False)
    return {**c, **kw}


def decode_case(name, **kw):
    c = dict(name=name, op="decode", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, N=1, prefix=1024, T=256, least=1, loose=0)
    return {**c, **kw}


def insert_case(name, **kw):
    c = dict(name=name, op="insert", dtype="bf16", B=4, Hkv=8, D=128, T=1024, n_sink=4, n_local=32)
    return {**c, **kw}


def compress_case(name, **kw):
    c = dict(name=name, op="compress", dtype="bf16", B=1, Hkv=8, D=128, S=8192, budget=1024, n_sink=4, n_local=64, least=1)
    return {**c, **kw}


def listed():
    return [
        # one decode token of 64 sequences at ragged positions up to 128K
        rotary_case("rotary step", B=64, theta=500000.0),
        # a 32K prompt, its queries and keys views of one packed projection, frequencies stretched by parts
        rotary_case("rotary prompt 32K", S=32768, theta=500000.0, scaling="turns", factor=8.0, packed=True),
        # the gradient of a training step in fp32: interleaved pairs over half of each head
        rotary_case("rotary gradient f32", dtype="f32", B=2, S=4099, Hq=16, Hkv=4, rot=64, layout="interleaved",
                    scaling="ramp", factor=4.0, orig=2048, amplitude=1.138629, gradient=True),
        # a few short conversations over a short system prompt: latency counts
        decode_case("decode 4 over 1K", B=4, Hq=16, Hkv=4, D=64, prefix=1021, T=65),
        # a serving batch over an 8K document
        decode_case("decode 32 over 8K", B=32, prefix=8192, T=1024),
        # three documents of different lengths, ragged groups, sequences without a prefix and an empty one
        decode_case("decode 3 prefixes", B=24, Hq=40, N=3, prefix=5000, T=777, least=0, loose=3),
        # many samples of one very long document: the batch shares its 128K tokens
        decode_case("decode 64 over 128K", B=64, prefix=131072, T=4096),
        # fp32 throughout
        decode_case("decode f32", dtype="f32", B=8, Hq=16, Hkv=4, prefix=4096, T=511),
        # the smallest full cache
        insert_case("insert 4 x 257", B=4, Hkv=4, D=64, T=257),
        # a serving batch with 4K-token caches
        insert_case("insert 64 x 4096", B=64, T=4096),
        # a batch of ragged prompts into 1K caches
        compress_case("compress 8K to 1K", B=8),
        # one 128K prompt into an 8K cache
        compress_case("compress 128K to 8K", S=131072, budget=8192),
    ]


def span(rng, lo, hi):
    """An integer in [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "decode", "decode", "insert", "compress"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 256])
        layout = rng.choice(["half", "interleaved"])
        c = rotary_case("", dtype=rng.choice(["bf16", "bf16", "f32"]), B=span(rng, 1, 64), Hkv=Hkv,
                        Hq=Hkv * rng.randint(1, 8), D=D, rot=rng.choice([D, D, D // 2, D // 4]), layout=layout,
                        theta=rng.choice([10000.0, 500000.0, 1000000.0]), far=span(rng, 100, 1000000),
                        scaling=rng.choice(["none", "linear", "ntk", "turns", "ramp"]), orig=rng.choice([2048, 4096, 8192]),
                        packed=rng.random() < 0.4, gradient=rng.random() < 0.3)
        if c["scaling"] != "none":
            c["factor"] = rng.choice([2.0, 4.0, 8.0, 32.0])
        most = 32768 * 40 * 128 * 2 // (c["B"] * (c["Hq"] + Hkv) * D * SIZE[c["dtype"]])
        c["S"] = span(rng, 1, max(1, most))
    elif op == "decode":
        f32 = rng.random() < 0.25
        c = decode_case("", dtype="f32" if f32 else "bf16", B=span(rng, 1, 16 if f32 else 64), Hkv=Hkv,
                        Hq=Hkv * rng.randint(1, 8), D=rng.choice([64, 128]), N=rng.choice([0, 1, 1, 1, 2, 4]),
                        prefix=span(rng, 1, 8192 if f32 else 131072), T=span(rng, 1, 1024 if f32 else 4096),
                        least=rng.randint(0, 1))
        if c["N"] > 1:
            c["prefix"] = max(1, c["prefix"] // c["N"])
        c["N"] = min(c["N"], c["B"])
        c["loose"] = rng.choice([0, 0, 1, 3]) if c["B"] - c["N"] >= 3 and c["N"] else 0
    elif op == "insert":
        c = insert_case("", dtype=rng.choice(["bf16", "bf16", "f32"]), B=span(rng, 1, 64), Hkv=Hkv,
                        D=rng.choice([64, 96, 128]), T=span(rng, 40, 4096), n_sink=rng.randint(0, 4), n_local=rng.randint(1, 32))
        if c["dtype"] == "f32":
            c["B"] = min(c["B"], 32)
    else:
        S = span(rng, 100, 131072)
        c = compress_case("", dtype=rng.choice(["bf16", "bf16", "f32"]), B=span(rng, 1, max(1, 131072 // S)), Hkv=Hkv,
                          D=rng.choice([64, 96, 128]), S=S, n_sink=rng.randint(0, 4), least=rng.randint(0, 1))
        c["budget"] = span(rng, 32, max(33, S // 8 if c["dtype"] == "bf16" else S // 16))
        c["n_local"] = rng.randint(0, c["budget"] // 2)
    c.pop("name")
    return c


# ------------------------------------------------------------------ inputs

def lengths(B, T, least, gen):
    """B lengths spread evenly over [least, T], in the seed's order."""
    at = torch.arange(B, dtype=torch.float64) / max(1, B - 1) if B > 1 else torch.ones(1, dtype=torch.float64)
    n = (least + (T - least) * at).round().to(torch.int32)
    return n[torch.randperm(B, generator=gen)]


def group_starts(c):
    """The first sequence of each prefix's group and the last one's end: ragged groups, `loose` sequences behind them."""
    n, N = c["B"] - c["loose"], c["N"]
    cut = [n * k * (k + 1) // (N * (N + 1)) if N > 1 else n * k for k in range(N + 1)]
    return [max(v, k) for k, v in enumerate(cut[:-1])] + [n] if N else [0]


def prefix_lengths(c):
    """Of N prefixes the first is whole, the others shorter."""
    return [max(1, c["prefix"] * (c["N"] - k) // c["N"] - 3 * k) for k in range(c["N"])]


def frequencies(c):
    """Radians a position, for each pair of the rotated part, in 64 bits."""
    rot, f = c["rot"], c["factor"]
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        return (c["theta"] * f ** (rot / (rot - 2))) ** (-i / rot) if rot > 2 else torch.ones(1, dtype=torch.float64)
    w = c["theta"] ** (-i / rot)
    if c["scaling"] == "linear":
        return w / f
    if c["scaling"] == "turns":  # pairs that turn often within the original length keep their frequency
        keep = ((c["orig"] * w / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return w / f * (1 - keep) + w * keep
    if c["scaling"] == "ramp":  # the same, the ramp over the pair's index
        at = [rot * math.log(c["orig"] / (t * 2 * math.pi)) / (2 * math.log(c["theta"])) for t in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        keep = 1 - ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w / f * (1 - keep) + w * keep
    return w


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 11)
    host = torch.Generator()
    host.manual_seed(seed * 104729 + 5)
    dt = DTYPE[c["dtype"]]

    def normal(*shape):
        """Standard normal values, made in the working type and slice by slice, so that large caches fit."""
        x = torch.empty(shape, dtype=dt, device="cuda")
        for part in x if x.numel() > 1 << 28 else [x]:
            part.normal_(generator=gen)
        return x

    s = {"case": c}
    if c["op"] == "rotary":
        B, S, D, Hq, Hkv = c["B"], c["S"], c["D"], c["Hq"], c["Hkv"]
        if c["packed"]:
            both = normal(B, S, (Hq + 2 * Hkv) * D)
            s["q"] = both[..., :Hq * D].view(B, S, Hq, D)
            s["k"] = both[..., Hq * D:(Hq + Hkv) * D].view(B, S, Hkv, D)
        else:
            s["q"], s["k"] = normal(B, S, Hq, D), normal(B, S, Hkv, D)
        first = torch.randint(0, max(1, c["far"] - S), (B, 1), generator=host)
        s["positions"] = (first + torch.arange(S)).to(torch.int32).cuda()
        s["freqs"] = frequencies(c).cuda()
        if own:
            from query_adaptive_chunk_b200.steps import Rotary
            s["rotary"] = Rotary(c["rot"], theta=c["theta"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                 orig_len=c["orig"], amplitude=c["amplitude"], device="cuda")
    elif c["op"] == "decode":
        B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
        s["q"] = normal(B, Hq, D)
        s["K"], s["V"] = normal(B, Hkv, T, D), normal(B, Hkv, T, D)
        s["len"] = lengths(B, T, c["least"], host).cuda()
        s["weights"] = torch.zeros(B, Hkv, T, device="cuda")  # the first step's sums
        if c["N"]:
            s["Kp"], s["Vp"] = normal(c["N"], Hkv, c["prefix"], D), normal(c["N"], Hkv, c["prefix"], D)
            # a document's first token draws much of the attention
            s["Kp"][:, :, 0] += 3 * s["q"][0, ::Hq // Hkv] / D ** 0.5
            s["prefix_len"] = torch.tensor(prefix_lengths(c), dtype=torch.int32).cuda()
            s["group_start"] = torch.tensor(group_starts(c), dtype=torch.int32).cuda()
            at = torch.arange(B).view(B, 1)
            start = torch.tensor(group_starts(c))
            s["member"] = ((at >= start[:-1]) & (at < start[1:])).cuda()  # [B, N]
        if own:
            from query_adaptive_chunk_b200.steps import SharedPrefixDecoder, TokenCache
            cache = TokenCache(s["K"], s["V"], lengths=s["len"], weights=s["weights"])
            s["decoder"] = SharedPrefixDecoder(cache, Hq=Hq, Kp=s.get("Kp"), Vp=s.get("Vp"), prefix_len=s.get("prefix_len"),
                                               group_start=s.get("group_start"), out_dtype=dt)
    else:
        B, Hkv, D = c["B"], c["Hkv"], c["D"]
        T = c["T"] if c["op"] == "insert" else c["S"]
        s["K"], s["V"] = normal(B, Hkv, T, D), normal(B, Hkv, T, D)
        # sums of attention weights: a few heavy tokens and a long tail; some tokens never attended to
        w = torch.rand(B, Hkv, T, generator=gen, device="cuda")
        s["weights"] = torch.where(w > 0.1, w ** 8 * 20, torch.zeros_like(w))
        if c["op"] == "insert":
            s["k"], s["v"] = normal(B, Hkv, D), normal(B, Hkv, D)
            s["len"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
            # the cache has evicted already: its slots hold T of the 2 T positions so far, in no order
            order = torch.rand(B, Hkv, T, generator=gen, device="cuda").argsort(-1)
            s["positions"] = (2 * order + (order >= T // 2)).to(torch.int32)
            s["next"] = torch.full((B,), 2 * T + 1, dtype=torch.int32, device="cuda")
            if own:
                from query_adaptive_chunk_b200.steps import TokenCache
                s["cache"] = TokenCache(s["K"], s["V"], lengths=s["len"], next_pos=s["next"], positions=s["positions"],
                                        weights=s["weights"], n_sink=c["n_sink"], n_local=c["n_local"])
        else:
            s["len"] = lengths(B, T, c["least"], host).cuda()
            n = c["budget"]
            s["Kc"], s["Vc"] = (torch.zeros(B, Hkv, n, D, dtype=dt, device="cuda") for _ in range(2))
            s["weights_c"] = torch.zeros(B, Hkv, n, device="cuda")
            s["positions_c"] = torch.zeros(B, Hkv, n, dtype=torch.int32, device="cuda")
            s["len_c"] = torch.zeros(B, dtype=torch.int32, device="cuda")
            if own:
                from query_adaptive_chunk_b200.steps import TokenCache
                s["cache"] = TokenCache(s["Kc"], s["Vc"], lengths=s["len_c"], positions=s["positions_c"],
                                        weights=s["weights_c"], n_sink=c["n_sink"], n_local=c["n_local"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"rotary": run_rotary, "decode": run_decode, "insert": run_insert, "compress": run_compress}[state["case"]["op"]](state)


def run_rotary(s):
    c = s["case"]
    if own:
        q, k = s["rotary"].rotate(s["q"], s["k"], positions=s["positions"], transpose=c["gradient"])
        return {"q": q, "k": k}
    t = s["positions"].double()[..., None] * s["freqs"]  # [B, S, rot/2]
    cos = (t.cos() * c["amplitude"]).float()[:, :, None]
    sin = (t.sin() * c["amplitude"]).float()[:, :, None]
    if c["gradient"]:
        sin = -sin

    def turn(x):
        rot, half = c["rot"], c["rot"] // 2
        r, rest = x[..., :rot].float(), x[..., rot:]
        if c["layout"] == "half":
            u, v = r[..., :half], r[..., half:]
            r = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        else:
            u, v = r[..., 0::2], r[..., 1::2]
            r = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        return torch.cat([r.to(x.dtype), rest], -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def run_decode(s):
    if own:
        out, lse = s["decoder"].attend(s["q"])
        return {"out": out, "lse": lse, "weights": s["weights"]}
    q, K, V = s["q"].float(), s["K"].float(), s["V"].float()
    B, Hkv, T, D = K.shape
    G = q.shape[1] // Hkv
    scale = 1.0 / math.sqrt(D)
    qg = q.view(B, Hkv, G, D)
    neg = float("-inf")
    hidden = torch.arange(T, device=q.device) >= s["len"].view(B, 1, 1, 1)
    so = (qg @ K.transpose(-1, -2) * scale).masked_fill(hidden, neg)  # [B, Hkv, G, T]
    m = so.amax(-1)
    if "Kp" in s:
        N, P = s["Kp"].shape[0], s["Kp"].shape[2]
        # every prefix's keys on one axis: [Hkv, N P, D]; a sequence sees its own prefix's
        kp = s["Kp"].float().transpose(0, 1).reshape(Hkv, N * P, D)
        vp = s["Vp"].float().transpose(0, 1).reshape(Hkv, N * P, D)
        qh = qg.transpose(0, 1).reshape(Hkv, B * G, D)
        seen = (torch.arange(P, device=q.device) < s["prefix_len"].view(N, 1)) & s["member"].view(B, N, 1)  # [B, N, P]
        sp = (qh @ kp.transpose(-1, -2) * scale).view(Hkv, B, G, N * P).masked_fill_(~seen.view(1, B, 1, N * P), neg)
        m = torch.maximum(m, sp.amax(-1).transpose(0, 1))
    base = m.clamp(min=-3e38)  # a row that sees nothing
    eo = (so - base[..., None]).exp()
    l, o = eo.sum(-1), eo @ V
    if "Kp" in s:
        ep = sp.sub_(base.transpose(0, 1)[..., None]).exp_()
        l = l + ep.sum(-1).transpose(0, 1)
        o = o + (ep.view(Hkv, B * G, N * P) @ vp).view(Hkv, B, G, D).transpose(0, 1)
    some = l > 0
    inv = torch.where(some, 1 / l, torch.zeros_like(l))[..., None]
    s["weights"] += torch.where(hidden[:, :, 0], 0.0, (eo * inv).sum(2))
    lse = torch.where(some, base + l.log(), neg)
    return {"out": (o * inv).reshape(B, Hkv * G, D).to(s["q"].dtype), "lse": lse.reshape(B, Hkv * G), "weights": s["weights"]}


def run_insert(s):
    c = s["case"]
    if own:
        s["cache"].insert(s["k"], s["v"])
    else:
        pos, nxt = s["positions"], s["next"].view(-1, 1, 1)
        fixed = (pos < c["n_sink"]) | (pos >= nxt - c["n_local"])
        w = s["weights"].masked_fill(fixed, float("inf"))
        # the lowest slot of those with the least weight
        slot = torch.where(w == w.amin(-1, keepdim=True), torch.arange(w.shape[-1], device=w.device), w.shape[-1]).amin(-1, keepdim=True)
        at = slot[..., None].expand(-1, -1, 1, c["D"])
        s["K"].scatter_(2, at, s["k"][:, :, None])
        s["V"].scatter_(2, at, s["v"][:, :, None])
        s["weights"].scatter_(2, slot, 0.0)
        s["positions"].scatter_(2, slot, nxt.expand(-1, w.shape[1], -1))
        s["next"] += 1
    return {"K": s["K"], "V": s["V"], "weights": s["weights"], "positions": s["positions"], "len": s["len"], "next": s["next"]}


def run_compress(s):
    c = s["case"]
    if own:
        s["cache"].compress(s["K"], s["V"], s["weights"], lengths=s["len"])
    else:
        B, Hkv, S, D = s["K"].shape
        n = c["budget"]
        row = torch.arange(S, device=s["K"].device)
        length = s["len"].view(B, 1, 1)
        fixed = (row < c["n_sink"]) | (row >= length - c["n_local"])
        w = s["weights"].masked_fill(fixed, float("inf")).masked_fill(row >= length, float("-inf"))
        # the heaviest n, the lower row first among equals; then in the order of their rows
        top = w.sort(dim=-1, descending=True, stable=True)[1][..., :n]
        kept = top < length
        top = torch.where(kept, top, S).sort(-1)[0]
        kept = top < length
        top = torch.where(kept, top, 0)
        at = top[..., None].expand(-1, -1, -1, D)
        s["Kc"].copy_(torch.where(kept[..., None], s["K"].gather(2, at), s["Kc"]))
        s["Vc"].copy_(torch.where(kept[..., None], s["V"].gather(2, at), s["Vc"]))
        s["weights_c"].copy_(torch.where(kept, s["weights"].gather(2, top), s["weights_c"]))
        s["positions_c"].copy_(torch.where(kept, top.to(torch.int32), s["positions_c"]))
        s["len_c"].copy_(s["len"].clamp(max=n))
    return {"K": s["Kc"], "V": s["Vc"], "weights": s["weights_c"], "positions": s["positions_c"], "len": s["len_c"]}


# ------------------------------------------------------------------ work

def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * e + 4 * c["B"] * c["S"], "flops": 6 * n // 2 * c["rot"] // c["D"]}
    if c["op"] == "decode":
        B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
        own_rows = int(lengths(B, c["T"], c["least"], torch.Generator()).sum())
        plen = prefix_lengths(c) if c["N"] else []
        start = group_starts(c)
        pairs = own_rows + sum(p * (start[n + 1] - start[n]) for n, p in enumerate(plen))
        rows = Hkv * (own_rows + sum(plen))
        return {"bytes": 2 * rows * D * e + 8 * Hkv * own_rows + 2 * B * Hq * D * e + 4 * B * Hq, "flops": 4 * pairs * Hq * D}
    if c["op"] == "insert":
        u = c["B"] * c["Hkv"]
        return {"bytes": u * (8 * c["T"] + 4 * c["D"] * e + 8), "flops": u * c["T"]}
    n = lengths(c["B"], c["S"], c["least"], torch.Generator())
    kept = c["Hkv"] * int(n.clamp(max=c["budget"]).sum())
    return {"bytes": 4 * c["Hkv"] * int(n.sum()) + kept * (4 * c["D"] * e + 8), "flops": c["Hkv"] * int(n.sum())}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        w = exact_frequencies(c)
        turn = torch.polar(torch.tensor(c["amplitude"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[..., None] * w * (-1 if c["gradient"] else 1))[:, :, None]

        def of(x):
            x = x.double()
            r = x[..., :c["rot"]]
            pairs = r.unflatten(-1, (2, -1)).transpose(-1, -2) if c["layout"] == "half" else r.unflatten(-1, (-1, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.transpose(-1, -2) if c["layout"] == "half" else z
            return torch.cat([z.flatten(-2), x[..., c["rot"]:]], -1)

        return {"q": of(s["q"]), "k": of(s["k"])}
    if c["op"] == "decode":
        B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
        G = Hq // Hkv
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64, device="cuda")
        weights = s["weights"].double()
        start, plen = group_starts(c), prefix_lengths(c) if c["N"] else []
        for b in range(B):
            n = int(s["len"][b])
            keys, values = [s["K"][b, :, :n]], [s["V"][b, :, :n]]
            for g, p in enumerate(plen):
                if start[g] <= b < start[g + 1]:
                    keys.append(s["Kp"][g, :, :p])
                    values.append(s["Vp"][g, :, :p])
            k, v = torch.cat(keys, 1).double(), torch.cat(values, 1).double()
            if k.shape[1] == 0:
                continue
            logits = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(Hkv, G, D), k) / math.sqrt(D)
            p = torch.softmax(logits, -1)
            out[b] = torch.einsum("hgt,htd->hgd", p, v).reshape(Hq, D)
            lse[b] = torch.logsumexp(logits, -1).reshape(Hq)
            weights[b, :, :n] += p[..., :n].sum(1)
        return {"out": out, "lse": lse, "weights": weights}
    if c["op"] == "insert":
        K, V, weights = s["K"].double(), s["V"].double(), s["weights"].double()
        pos, nxt = s["positions"], s["next"]
        for b in range(c["B"]):
            for h in range(c["Hkv"]):
                free = ((pos[b, h] >= c["n_sink"]) & (pos[b, h] < nxt[b] - c["n_local"])).nonzero()[:, 0]
                w = weights[b, h, free]
                at = free[(w == w.min()).nonzero()[0, 0]]
                K[b, h, at], V[b, h, at], weights[b, h, at], pos[b, h, at] = s["k"][b, h].double(), s["v"][b, h].double(), 0.0, nxt[b]
        return {"K": K, "V": V, "weights": weights, "positions": pos, "len": s["len"], "next": nxt + 1}
    K, V, weights = (torch.zeros_like(s[k], dtype=torch.float64) for k in ("Kc", "Vc", "weights_c"))
    pos = s["positions_c"]
    for b in range(c["B"]):
        n = int(s["len"][b])
        lo, hi = min(c["n_sink"], n), max(min(c["n_sink"], n), n - c["n_local"])
        free = max(0, min(n, c["budget"]) - lo - (n - hi))
        for h in range(c["Hkv"]):
            # by weight from the heaviest, then by row: numbers of (-weight, row) in order
            best = torch.argsort(-s["weights"][b, h, lo:hi].double(), stable=True)[:free] + lo
            kept = torch.cat([torch.arange(lo, device="cuda"), best, torch.arange(hi, n, device="cuda")]).sort()[0][:c["budget"]]
            m = len(kept)
            K[b, h, :m], V[b, h, :m] = s["K"][b, h, kept].double(), s["V"][b, h, kept].double()
            weights[b, h, :m], pos[b, h, :m] = s["weights"][b, h, kept].double(), kept.to(torch.int32)
        s["len_c"][b] = min(n, c["budget"])
    return {"K": K, "V": V, "weights": weights, "positions": pos, "len": s["len_c"]}


def exact_frequencies(c):
    """As frequencies(), pair by pair."""
    w = []
    for i in range(c["rot"] // 2):
        e = 2.0 * i / c["rot"]
        base = c["theta"] ** -e
        if c["scaling"] == "linear":
            base = base / c["factor"]
        elif c["scaling"] == "ntk":
            base = base * c["factor"] ** (-2.0 * i / (c["rot"] - 2)) if c["rot"] > 2 else 1.0
        elif c["scaling"] in ("turns", "ramp"):
            if c["scaling"] == "turns":
                keep = (c["orig"] / (2 * math.pi / base) - 1.0) / 31.0
            else:
                lo = max(0, math.floor(c["rot"] / 2 * math.log(c["orig"] / (64 * math.pi), c["theta"])))
                hi = min(c["rot"] - 1, math.ceil(c["rot"] / 2 * math.log(c["orig"] / (2 * math.pi), c["theta"])))
                keep = 1.0 - (i - lo) / max(hi - lo, 0.001)
            keep = min(1.0, max(0.0, keep))
            base = base * (keep + (1.0 - keep) / c["factor"])
        w.append(base)
    return torch.tensor(w, dtype=torch.float64, device="cuda")
