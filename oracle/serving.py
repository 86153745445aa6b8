"""CPU oracle of the serving operators (fp64, plain numpy): rotary positions,
decode over shared prefixes with attention-weight sums, and the cache that is
bounded by those sums.

TEST INFRASTRUCTURE, as ``csa_oracle``: only tests import it, and it shares no
code with the library.  Arrays come in as fp64 (bf16 values are exact).
"""
from __future__ import annotations

import math

import numpy as np


def rotary_freqs(rot, theta, scaling="none", factor=1.0, orig_len=8192.0, low=1.0, high=32.0):
    """Radians per position of the rot/2 pairs."""
    out = []
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "ntk":
            w = (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) if rot > 2 else 1.0
        elif scaling in ("turns", "ramp"):
            if scaling == "turns":
                keep = (orig_len * w / (2 * math.pi) - low) / (high - low)
            else:
                def dim(turns):
                    return rot * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(theta))
                lo, hi = max(0, math.floor(dim(high))), min(rot - 1, math.ceil(dim(low)))
                keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            keep = min(1.0, max(0.0, keep))
            w = (1.0 - keep) * w / factor + keep * w
        out.append(w)
    return np.array(out)


def rotary(x, positions, freqs, layout="half", amplitude=1.0, transpose=False):
    """x [B, S, H, D], positions [B, S] -> the turned x."""
    rot = 2 * len(freqs)
    t = np.asarray(positions, dtype=np.float64)[:, :, None, None] * freqs
    c, s = amplitude * np.cos(t), amplitude * np.sin(t) * (-1.0 if transpose else 1.0)
    y = np.array(x, dtype=np.float64)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def prefix_decode(q, K, V, lengths, scale, Kp=None, Vp=None, prefix_len=None, group_start=None,
                  weights=None, decay=1.0):
    """q [B, Hq, D], K/V [B, Hkv, T, D], Kp/Vp [N, Hkv, Tp, D].  Returns out [B, Hq,
    D], lse [B, Hq], the new weights [B, Hkv, T] (or None), and spread [B, Hq, D] =
    sum_j p_j |v_j| (what a relative rounding of the p_j is a share of)."""
    B, Hq, D = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    out, spread, lse = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    new = None if weights is None else np.array(weights, dtype=np.float64)
    for b in range(B):
        n = int(lengths[b])
        g = -1
        for i in range(0 if Kp is None else len(Kp)):
            if group_start[i] <= b < group_start[i + 1]:
                g = i
        for h in range(Hkv):
            k, v = K[b, h, :n], V[b, h, :n]
            if g >= 0:
                k = np.concatenate([k, Kp[g, h, :prefix_len[g]]])
                v = np.concatenate([v, Vp[g, h, :prefix_len[g]]])
            total = np.zeros(n)
            for hq in range(h * G, (h + 1) * G):
                if len(k) == 0:
                    continue
                s = scale * (k @ q[b, hq])
                m = s.max()
                e = np.exp(s - m)
                lse[b, hq] = m + math.log(e.sum())
                p = e / e.sum()
                out[b, hq], spread[b, hq] = p @ v, p @ np.abs(v)
                total += p[:n]
            if new is not None:
                new[b, h, :n] = (decay * new[b, h, :n] if decay else 0.0) + total
    return out, lse, new, spread


def _rank(w):
    """A weight as a comparable number: NaN as -inf."""
    return -math.inf if math.isnan(w) else float(w)


def cache_insert(cache, k, v, budget, n_sink, n_local):
    """cache: dict of K, V, weights, positions, lengths, next_pos (changed in
    place); k, v [B, Hkv, D].  Returns the slot of each (b, h), -1 if none."""
    B, Hkv, _ = k.shape
    slots = -np.ones((B, Hkv), dtype=int)
    for b in range(B):
        n, p = int(cache["lengths"][b]), int(cache["next_pos"][b])
        if p < 0:
            continue
        for h in range(Hkv):
            slot = n
            if n == budget:
                slot, best = -1, None
                for j in range(n):
                    at = int(cache["positions"][b, h, j])
                    if at < n_sink or at >= p - n_local:
                        continue
                    w = _rank(cache["weights"][b, h, j])
                    if best is None or w < best:
                        slot, best = j, w
            slots[b, h] = slot
            cache["K"][b, h, slot], cache["V"][b, h, slot] = k[b, h], v[b, h]
            cache["weights"][b, h, slot], cache["positions"][b, h, slot] = 0.0, p
        cache["lengths"][b], cache["next_pos"][b] = min(n + 1, budget), p + 1
    return slots


def cache_compress(weights, lengths, budget, n_sink, n_local, positions=None, next_pos=None):
    """The kept rows of each (b, h), ascending: [B][Hkv] lists."""
    B, Hkv, _ = weights.shape
    kept = []
    for b in range(B):
        n = int(lengths[b])
        heads = []
        for h in range(Hkv):
            nxt = n if next_pos is None else int(next_pos[b])
            if nxt < 0:  # inactive: it stands behind its last row
                nxt = n if positions is None else 1 + max((int(x) for x in positions[b, h, :n]), default=0)
            order = []
            for j in range(n):
                at = j if positions is None else int(positions[b, h, j])
                fixed = at < n_sink or at >= nxt - n_local
                order.append((0 if fixed else 1, -_rank(weights[b, h, j]) if not fixed else 0.0, j))
            heads.append(sorted(j for _, _, j in sorted(order)[:budget]))
        kept.append(heads)
    return kept
