"""Decode and prefill steps assembled from the C-ABI calls.

``SparseDecoder`` owns the buffers of one decode configuration (chunk
summaries, scores, index lists, split-K partials, outputs) and runs a step
as: score -> select (top-k / top-p / hierarchical) -> sparse decode ->
LSE merge.  ``BlockSparsePrefill`` runs tile means -> causal scores -> top-k
-> block-sparse prefill.  ``Rotary``, ``TokenCache`` and ``SharedPrefixDecoder``
serve sequences that share prefixes: positions, a cache of their own bounded
by attention weight, and the decode over both.  Buffers come from torch (device
memory); every computation is a call into libcsa.
"""
from __future__ import annotations

import math

import torch

from . import csa


def _dt(t: torch.Tensor) -> int:
    return csa.CSA_BF16 if t.dtype == torch.bfloat16 else csa.CSA_F32


class SparseDecoder:
    """Query-adaptive chunk-sparse decode over a fixed KV cache.

    K, V: [B, Hkv, T, D] (bf16 or fp32, contiguous, on the current device).
    select: "topk" | "topk_union" (per-head top-k, GQA union) | "topp" | "hier".  The summaries (and meta-summaries)
    are computed once here, as part of building the cache.  With fused=True
    (default) a step is two launches: fused score+select (one CTA per unit)
    and the merged split-K decode; fused=False runs the separate calls
    (score, select, decode, merge).  With a bf16 cache and fused=True,
    ``step`` is one call of csa_decode_step, whose decode streams the
    full-attention heads while the selection runs.

    hybrid=True (bf16, fused): every sparse head also attends over gist
    key/value rows (the hybrid context of SSA): those of its selected chunks
    (gist_scope="selected", the method section's reading) or of every chunk
    (gist_scope="all").  gist=(Kg, Vg), each [B, Hkv, T/L, D] bf16, is the
    model's gist KV; when it is not given the rows are built here with the
    cache, as the chunk means of K and V in bf16 (a stand-in).

    rope_theta > 0 (the RoPE-aware split): K and the queries given to ``step``
    are pre-RoPE; chunks are scored on them, and attention runs on rotated
    copies (csa_rope): the cache is rotated once here (positions 0..T-1) and
    each step rotates its query at position T - 1."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, *, Hq: int, L: int, select: str,
                 n_sink: int, n_local: int, k_free: int = 0, proj: torch.Tensor | None = None,
                 p: float = 0.9, budget: int = 256, full_heads=(), Gm: int = 0, top_meta: int = 0,
                 scale: float | None = None, num_parts: int = 0, out_dtype=torch.float32,
                 fused: bool = True, hybrid: bool = False, gist=None, gist_scope: str = "selected",
                 rope_theta: float = 0.0):
        assert K.is_contiguous() and V.is_contiguous() and K.shape == V.shape
        self.K, self.V = K, V
        B, Hkv, T, D = K.shape
        self.B, self.Hq, self.Hkv, self.T, self.D, self.L = B, Hq, Hkv, T, D, L
        self.C = T // L
        self.select, self.n_sink, self.n_local, self.k_free = select, n_sink, n_local, k_free
        self.p, self.budget, self.Gm, self.top_meta = p, budget, Gm, top_meta
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.proj = proj
        self.R = 0 if proj is None else proj.shape[1]
        self.dtype = _dt(K)
        dev = K.device
        U = B * Hkv
        Ds = self.R if proj is not None else D
        self.summ = torch.empty(B, Hkv, self.C, Ds, dtype=torch.float32, device=dev)
        csa.csa_chunk_summaries(K, self.dtype, B, Hkv, T, D, L, proj, self.R, self.summ)
        self.meta = None
        if select == "hier":
            self.meta = torch.empty(B, Hkv, self.C // Gm, Ds, dtype=torch.float32, device=dev)
            csa.csa_meta_summaries(self.summ, B, Hkv, self.C, Ds, Gm, self.meta)
        self.rope_theta = float(rope_theta)
        self.K_att, self.q_rot = K, None
        if self.rope_theta > 0:
            assert not hybrid, "the hybrid context is not combined with RoPE here"
            self.K_att = torch.empty_like(K)
            csa.csa_rope(K, self.K_att, self.dtype, B * Hkv * T, D, T, 0, self.rope_theta)
            self.q_rot = torch.empty(B, Hq, D, dtype=K.dtype, device=dev)
        self.Kg = self.Vg = None
        self.gist_scope = gist_scope
        if hybrid and gist is not None:
            assert fused and K.dtype == torch.bfloat16, "the hybrid context needs a fused bf16 decode"
            self.Kg, self.Vg = gist
        elif hybrid:
            assert fused and K.dtype == torch.bfloat16, "the hybrid context needs a fused bf16 decode"
            means = torch.empty(B, Hkv, self.C, D, dtype=torch.float32, device=dev)
            csa.csa_chunk_summaries(K, self.dtype, B, Hkv, T, D, L, None, 0, means)
            self.Kg = means.to(torch.bfloat16)
            csa.csa_chunk_summaries(V, self.dtype, B, Hkv, T, D, L, None, 0, means)
            self.Vg = means.to(torch.bfloat16)
        self.head_full = None
        if full_heads:
            hf = torch.zeros(Hkv, dtype=torch.uint8)
            hf[list(full_heads)] = 1
            self.head_full = hf.to(dev)
        extra = budget if select == "topp" else k_free
        if select == "topk_union":
            extra = (Hq // Hkv) * k_free
        self.kmax = min(self.C, extra + n_sink + n_local)
        self.scores = torch.zeros(B, Hkv, 1, self.C, dtype=torch.float32, device=dev)
        self.idx = torch.full((U, self.kmax), -1, dtype=torch.int32, device=dev)
        self.count = torch.zeros(U, dtype=torch.int32, device=dev)
        self.n_p = torch.zeros(U, dtype=torch.int32, device=dev)
        self.P = num_parts if num_parts > 0 else csa.csa_decode_default_parts(self.dtype, D, L)
        self.max_splits = self.P
        self.o_part = torch.empty(B, Hq, self.max_splits, D, dtype=torch.float32, device=dev)
        self.lse_part = torch.empty(B, Hq, self.max_splits, dtype=torch.float32, device=dev)
        self.out = torch.empty(B, Hq, D, dtype=out_dtype, device=dev)
        self.lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
        self.fused = fused
        self.num_parts = num_parts
        if fused:
            # sized for the larger of the two P the merged paths may use
            self.ws_bytes = max(csa.csa_decode_workspace_bytes(B, Hq, Hkv, D, self.P),
                                csa.csa_decode_workspace_bytes(B, Hq, Hkv, D, num_parts))
            self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.desc = None
        self.q_dev = None  # the device query buffer of step_host, made on first use
        if fused and self.dtype == csa.CSA_BF16:
            mode = {"topk": csa.CSA_SELECT_TOPK, "topp": csa.CSA_SELECT_TOPP,
                    "hier": csa.CSA_SELECT_HIER, "topk_union": csa.CSA_SELECT_TOPK_UNION}[select]
            self.desc = csa.decode_step_desc(
                K=self.K_att, V=V, B=B, Hq=Hq, Hkv=Hkv, D=D, T=T, L=L, scale=self.scale,
                head_full=self.head_full, mode=mode, summ=self.summ, proj=proj, R=self.R,
                meta=self.meta, Gm=Gm, top_meta=top_meta, k_free=k_free, n_sink=n_sink,
                n_local=n_local, logit_scale=1.0 / math.sqrt(D), p=p, budget=budget, idx=self.idx,
                count=self.count, kmax=self.kmax, n_p_out=self.n_p, num_parts=num_parts,
                workspace=self.workspace, workspace_bytes=self.ws_bytes, out=self.out,
                out_dtype=self.out.dtype, lse_out=self.lse, Kg=self.Kg, Vg=self.Vg,
                gist_scope=gist_scope)

    def select_chunks(self, q: torch.Tensor, stream=None):
        """Score + select: fills self.idx / self.count (and self.n_p for top-p)."""
        B, Hq, Hkv, D, C = self.B, self.Hq, self.Hkv, self.D, self.C
        U = B * Hkv
        qd = _dt(q)
        if self.select == "hier":
            csa.csa_select_hier(q, qd, self.meta, self.summ, B, Hq, Hkv, D, C, self.Gm,
                                self.top_meta, self.k_free, self.n_sink, self.n_local, self.idx,
                                self.count, self.kmax, stream=stream)
            return
        if self.fused and self.select == "topk":
            csa.csa_score_select_topk(q, qd, self.proj, self.R, self.summ, B, Hq, Hkv, D, C,
                                      self.head_full, self.k_free, self.n_sink, self.n_local,
                                      self.idx, self.count, self.kmax, stream=stream)
            return
        if self.select == "topk_union":  # one call: per-head scores never leave the SM
            csa.csa_score_select_topk_union(q, qd, self.proj, self.R, self.summ, B, Hq, Hkv, D, C,
                                            self.head_full, self.k_free, self.n_sink,
                                            self.n_local, self.idx, self.count, self.kmax,
                                            stream=stream)
            return
        if self.fused and self.select == "topp":
            csa.csa_score_select_topp(q, qd, self.proj, self.R, self.summ, B, Hq, Hkv, D, C,
                                      self.head_full, 1.0 / math.sqrt(D), self.p, self.budget,
                                      self.n_sink, self.n_local, self.idx, self.count, self.kmax,
                                      self.n_p, stream=stream)
            return
        csa.csa_score_chunks(q, qd, self.proj, self.R, self.summ, B, 1, Hq, Hkv, D, C,
                             self.head_full, 0, 0, self.scores, stream=stream)
        if self.select == "topk":
            csa.csa_select_topk(self.scores, U, C, None, self.k_free, self.n_sink, self.n_local,
                                self.idx, self.count, self.kmax, stream=stream)
        elif self.select == "topp":
            csa.csa_select_topp(self.scores, U, C, 1.0 / math.sqrt(D), self.p, self.budget,
                                self.n_sink, self.n_local, self.idx, self.count, self.kmax,
                                self.n_p, stream=stream)
        else:
            raise ValueError(self.select)

    def attend(self, q: torch.Tensor, stream=None):
        """Sparse split-K decode over the current index lists, then the LSE merge
        (one launch when fused)."""
        if self.Kg is not None:
            csa.csa_sparse_decode_merged_hybrid(q, self.K_att, self.V, self.Kg, self.Vg,
                                                self.gist_scope, self.dtype,
                                                self.idx, self.count, self.kmax, self.head_full,
                                                self.B, self.Hq, self.Hkv, self.D, self.T, self.L,
                                                self.scale, self.num_parts, self.workspace,
                                                self.ws_bytes, self.out, _dt(self.out), self.lse,
                                                stream=stream)
            return
        if self.fused:
            csa.csa_sparse_decode_merged(q, self.K_att, self.V, self.dtype, self.idx, self.count,
                                         self.kmax, self.head_full, self.B, self.Hq, self.Hkv,
                                         self.D, self.T, self.L, self.scale, self.num_parts,
                                         self.workspace, self.ws_bytes, self.out, _dt(self.out),
                                         self.lse, stream=stream)
            return
        csa.csa_sparse_decode(q, self.K_att, self.V, self.dtype, self.idx, self.count, self.kmax,
                              self.head_full, self.B, self.Hq, self.Hkv, self.D, self.T, self.L,
                              self.scale, self.P, self.max_splits, self.o_part, self.lse_part,
                              stream=stream)
        csa.csa_lse_merge(self.o_part, self.lse_part, self.B * self.Hq, self.max_splits, self.D,
                          self.out, _dt(self.out), self.lse, stream=stream)

    def step(self, q: torch.Tensor, stream=None):
        qa = q  # the query attention runs with
        if self.q_rot is not None:
            csa.csa_rope(q, self.q_rot, self.dtype, self.B * self.Hq, self.D, 1, self.T - 1,
                         self.rope_theta, stream=stream)
            qa = self.q_rot
        if self.desc is not None and q.dtype == torch.bfloat16:
            self.desc.q = qa.data_ptr()
            self.desc.q_score = q.data_ptr() if self.q_rot is not None else None
            csa.csa_decode_step(self.desc, stream=stream)
            return self.out, self.lse
        self.select_chunks(q, stream)
        self.attend(qa, stream)
        return self.out, self.lse

    def step_host(self, q_host: torch.Tensor, out_host: torch.Tensor,
                  lse_host: torch.Tensor | None = None, stream=None):
        """One step whose query and result live in pinned host memory
        (csa_decode_step_host): q_host [B, Hq, D] bf16 is copied into the
        decoder's own device query buffer, the step runs, and the output
        (and lse, when lse_host is given) are copied into out_host, all
        asynchronously on `stream`: synchronise it before reading out_host.
        Needs the one-call bf16 step without RoPE."""
        if self.desc is None or self.q_rot is not None:
            raise ValueError("step_host needs a fused bf16 decoder without RoPE")
        if self.q_dev is None:
            self.q_dev = torch.empty(self.B, self.Hq, self.D, dtype=torch.bfloat16,
                                     device=self.out.device)
        self.desc.q = self.q_dev.data_ptr()
        self.desc.q_score = None
        csa.csa_decode_step_host(self.desc, q_host, out_host, lse_host, stream=stream)

    def host_step_graph(self, q_host: torch.Tensor, out_host: torch.Tensor,
                        lse_host: torch.Tensor | None = None) -> "torch.cuda.CUDAGraph":
        """``step_host`` on these host buffers captured as a CUDA graph: each
        ``replay()`` copies the current contents of q_host in, runs the step
        and copies the result out (synchronise before reading out_host)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step_host(q_host, out_host, lse_host)  # warm the capture stream
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            self.step_host(q_host, out_host, lse_host)
        return g


class BlockSparsePrefill:
    """Block-sparse causal prefill: per (tile, KV head) the top-k_free chunks by
    tile-mean score plus the sink and the diagonal chunk."""

    def __init__(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, *, tile_m: int, L: int,
                 k_free: int, n_sink: int = 1, n_local: int = 1, scale: float | None = None):
        B, S, Hq, D = Q.shape
        Hkv = K.shape[1]
        self.Q, self.K, self.V = Q, K, V
        self.B, self.S, self.Hq, self.Hkv, self.D = B, S, Hq, Hkv, D
        self.tile_m, self.L, self.k_free, self.n_sink, self.n_local = tile_m, L, k_free, n_sink, n_local
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.n_tiles = S // tile_m
        self.C = S // L
        dev = Q.device
        self.kmax = min(self.C, k_free + n_sink + n_local)
        self.summ = torch.empty(B, Hkv, self.C, D, dtype=torch.float32, device=dev)
        csa.csa_chunk_summaries(K, _dt(K), B, Hkv, S, D, L, None, 0, self.summ)
        self.qbar = torch.empty(B, self.n_tiles, Hq, D, dtype=torch.float32, device=dev)
        self.scores = torch.empty(B, Hkv, self.n_tiles, self.C, dtype=torch.float32, device=dev)
        U = B * Hkv * self.n_tiles
        self.idx = torch.full((U, self.kmax), -1, dtype=torch.int32, device=dev)
        self.count = torch.zeros(U, dtype=torch.int32, device=dev)
        self.O = torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=dev)

    def select_chunks(self, stream=None):
        B, S, Hq, Hkv, D = self.B, self.S, self.Hq, self.Hkv, self.D
        csa.csa_tile_mean_q(self.Q, _dt(self.Q), B, S, Hq, D, self.tile_m, self.qbar, stream=stream)
        csa.csa_score_chunks(self.qbar, csa.CSA_F32, None, 0, self.summ, B, self.n_tiles, Hq, Hkv,
                             D, self.C, None, self.tile_m, self.L, self.scores, stream=stream)
        csa.csa_select_topk_causal(self.scores, B * Hkv * self.n_tiles, self.C, self.n_tiles,
                                   self.tile_m, self.L, self.k_free, self.n_sink, self.n_local,
                                   self.idx, self.count, self.kmax, stream=stream)

    def attend(self, stream=None):
        csa.csa_block_sparse_prefill(self.Q, self.K, self.V, self.idx, self.count, self.kmax,
                                     self.B, self.S, self.Hq, self.Hkv, self.D, self.tile_m,
                                     self.L, self.scale, self.O, stream=stream)

    def step(self, stream=None):
        self.select_chunks(stream)
        self.attend(stream)
        return self.O


def _bad(why: str):
    raise csa.CsaError(1, why)


_TYPES = (torch.bfloat16, torch.float32)


def _typed(name, dtype):
    if dtype not in _TYPES:
        _bad(f"{name} must be bf16 or fp32, not {dtype}")


def _empty_like(t, stream):
    """An output for a call on `stream`: allocated on it, so that its memory is
    not one that other streams' pending work still uses."""
    if stream is None:
        return torch.empty_like(t)
    if not isinstance(stream, torch.cuda.Stream):
        _bad("give the outputs with a raw stream")
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            _bad(f"{name} is on {t.device}, not {device}")


def _rows(name, t, dtype, shape=None):
    """A tensor whose last index is dense: its other strides, in elements."""
    if t.dtype != dtype:
        _bad(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        _bad(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        _bad(f"{name}: the last index must be dense")
    return st[:-1]


def _dense(name, t, dtype, shape):
    if t.dtype != dtype:
        _bad(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        _bad(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous")
    return t


def _wide_rows(name, t):
    """What the decode's 16-byte accesses need of a cache or prefix [n0, n1, rows, D]."""
    es = t.element_size()
    if t.data_ptr() % 16 or any(s * es % 16 for n, s in zip(t.shape[:3], t.stride()) if n > 1):
        _bad(f"{name}: rows must start on 16 bytes")
    if t.shape[2] > 1 and t.stride(2) < t.shape[3]:
        _bad(f"{name}: strides of the tokens must be at least D")


class _Turn(torch.autograd.Function):
    """Rotary.rotate for autograd: linear, so the gradient is the transposed
    rotation of the outputs' (and in its turn differentiable)."""

    @staticmethod
    def forward(ctx, rotary, transpose, pos0, positions, q, k):
        ctx.set_materialize_grads(False)
        # the positions of the forward pass, whatever becomes of the caller's (a
        # cache's next_pos advances in place)
        ctx.rotary, ctx.transpose, ctx.pos0 = rotary, transpose, pos0
        ctx.positions = None if positions is None else positions.clone()
        return rotary.rotate(q, k, positions=positions, pos0=pos0, transpose=transpose)

    @staticmethod
    def backward(ctx, *grads):
        out = [None, None]
        need = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[4 + i]]
        if need:
            # any strides and offset may come back (of an expanded sum: all zero)
            gs = [grads[i] if grads[i].stride(-1) == 1
                  and all(s % 2 == 0 for s in (*grads[i].stride()[:-1], grads[i].storage_offset()))
                  else grads[i].clone(memory_format=torch.contiguous_format) for i in need]
            y = ctx.rotary.rotate(*gs, positions=ctx.positions, pos0=ctx.pos0, transpose=not ctx.transpose)
            for i, g in zip(need, y if len(need) == 2 else (y,)):
                out[i] = g
        return None, None, None, None, *out


class Rotary:
    """Rotary positions (csa_rotary) with one frequency table.

    rot: values of each head that turn (the rest is copied); layout "half" or
    "interleaved" pairs; scaling "none", "linear", "ntk", "turns" or "ramp"
    with `factor` (and orig_len, low, high), or ``freqs`` (rot/2 fp64 radians per
    position) for any other rule; amplitude multiplies the turned values."""

    def __init__(self, rot: int, *, theta: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, orig_len: float = 8192,
                 low: float = 1.0, high: float = 32.0, amplitude: float = 1.0,
                 freqs: torch.Tensor | None = None, device="cuda"):
        self.rot, self.layout, self.amplitude = rot, csa._ROTARY_LAYOUT[layout], float(amplitude)
        self.table = torch.empty(rot // 2, dtype=torch.int64, device=device)
        if freqs is not None:
            freqs = _dense("freqs", freqs, torch.float64, (rot // 2,))
        self.table_ptr = self.table.data_ptr()
        with torch.cuda.device(self.table.device):
            csa.csa_rotary_table(rot, theta, scaling, factor, orig_len, low, high, freqs,
                                 self.table)

    def rotate(self, q: torch.Tensor, k: torch.Tensor | None = None, *,
               positions: torch.Tensor | None = None, pos0: int = 0, q_out=None, k_out=None,
               transpose: bool = False, stream=None):
        """Turns q [B, S, Hq, D] and k [B, S, Hkv, D] (any strides, the last
        index dense; a decode step has S = 1) in one launch.  positions: int32
        [B, S] (rows may repeat: expand a [1, S]), else pos0 + s.  Results go to
        q_out / k_out (q_out=q: in place), by default new tensors of `stream`
        (then a torch stream).
        transpose=True gives the gradient of the input from that of the output; autograd
        finds it by itself through q and k that require gradients, on the current
        stream and with new outputs (anything else is refused then).
        Returns (q_out, k_out), or q_out alone without k."""
        if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
            if q_out is not None or k_out is not None or stream is not None:
                _bad("q or k requires a gradient: no q_out, k_out or stream (detach them, or use torch.no_grad)")
            return _Turn.apply(self, transpose, pos0, positions, q, k)
        B, S, Hq, D = q.shape
        dt, dev = q.dtype, self.table.device
        if dt not in _TYPES:
            _typed("q", dt)
        if q_out is None:
            q_out = _empty_like(q, stream)
        x = (q.data_ptr(), q_out.data_ptr(), Hq, _rows("q", q, dt),
             _rows("q_out", q_out, dt, q.shape))
        x2 = (0, 0, 0, (0, 0, 0), (0, 0, 0))
        if k is not None:
            if k_out is None:
                k_out = _empty_like(k, stream)
            Hkv = k.shape[2]
            x2 = (k.data_ptr(), k_out.data_ptr(), Hkv, _rows("k", k, dt, (B, S, Hkv, D)),
                  _rows("k_out", k_out, dt, k.shape))
            if k.device != dev or k_out.device != dev:
                _bad(f"k and k_out must be on {dev}")
        pos = stride = 0
        if positions is not None:
            if positions.dtype != torch.int32 or positions.shape != (B, S) or positions.device != dev:
                _bad(f"positions must be int32 of shape {(B, S)} on {dev}")
            stride, s1 = positions.stride()
            if S > 1 and s1 != 1:
                _bad("positions: the token index must be dense")
            pos = positions.data_ptr()
        if q.device != dev or q_out.device != dev:
            _bad(f"q and q_out must be on {dev}")
        csa.csa_rotary(csa.ROTARY_PACK.pack(
            x[0], x[1], x[2], *x[3], *x[4], x2[0], x2[1], x2[2], *x2[3], *x2[4], csa._dt(dt), B, S, D,
            self.rot, self.layout, transpose, self.table_ptr, self.amplitude, pos, stride, pos0), stream)
        return q_out if k is None else (q_out, k_out)


class TokenCache:
    """A KV cache bounded by accumulated attention weight (csa_cache_insert,
    csa_cache_compress).

    K, V: [B, Hkv, T, D] bf16 or fp32, any strides with the last index dense
    ([B, T, Hkv, D] storage as a transposed view).  lengths [B] int32 slots in
    use, next_pos [B] int32 (the next token's position; negative: inactive),
    positions [B, Hkv, T] int32 and weights [B, Hkv, T] fp32: made here (empty
    cache, positions from 0) unless given; all are updated in place.  Slots are
    in no order; ``positions`` says where each token stands.  budget: slots kept
    (default T), the protected first n_sink positions and last n_local tokens
    among them."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, *, lengths=None, next_pos=None,
                 positions=None, weights=None, budget: int | None = None, n_sink: int = 0,
                 n_local: int = 0):
        B, Hkv, T, D = K.shape
        dev = K.device
        _typed("K", K.dtype)

        def own(name, t, dtype, shape):
            return torch.zeros(shape, dtype=dtype, device=dev) if t is None else _dense(name, t, dtype, shape)

        self.K, self.V, self.B, self.Hkv, self.T, self.D = K, V, B, Hkv, T, D
        self.lengths = own("lengths", lengths, torch.int32, (B,))
        self.next_pos = own("next_pos", next_pos, torch.int32, (B,))
        self.positions = own("positions", positions, torch.int32, (B, Hkv, T))
        self.weights = own("weights", weights, torch.float32, (B, Hkv, T))
        self.counters = torch.zeros(B, dtype=torch.int32, device=dev)
        self.budget = T if budget is None else budget
        self.k_stride, self.v_stride = _rows("K", K, K.dtype), _rows("V", V, K.dtype, K.shape)
        _same_device(dev, V=V, lengths=lengths, next_pos=next_pos, positions=positions, weights=weights)
        self.desc = csa.cache_desc(
            K=K, V=V, dtype=K.dtype, B=B, Hkv=Hkv, D=D, T=T, k_stride=self.k_stride,
            v_stride=self.v_stride, weights=self.weights, positions=self.positions,
            len=self.lengths, next_pos=self.next_pos, budget=self.budget, n_sink=n_sink,
            n_local=n_local, counters=self.counters)

    def insert(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """One new token per active sequence, k and v [B, Hkv, D] (the last
        index dense): into the next free slot, or over the lightest unprotected."""
        shape, dt = (self.B, self.Hkv, self.D), self.K.dtype
        csa.csa_cache_insert(self.desc, k, _rows("k", k, dt, shape), v, _rows("v", v, dt, shape),
                             stream=stream)

    def compress(self, K: torch.Tensor, V: torch.Tensor, weights: torch.Tensor, *, lengths=None,
                 positions=None, next_pos=None, stream=None):
        """Fills this cache from longer K, V [B, Hkv, S, D] with weights [B, Hkv,
        S] (a prompt's, as csa_token_importance gives them, or another cache's):
        all rows below `lengths`, or the protected and the heaviest ones up to
        the budget, in row order.  positions [B, Hkv, S] with next_pos [B], else
        the row numbers.  A sequence with a negative next_pos stays inactive."""
        B, Hkv, S, D = K.shape
        if (B, Hkv, D) != (self.B, self.Hkv, self.D):
            _bad("source K has other sizes than the cache")
        src = csa.cache_source(
            K=K, V=V, S=S, k_stride=_rows("source K", K, self.K.dtype),
            v_stride=_rows("source V", V, self.K.dtype, K.shape),
            weights=_dense("source weights", weights, torch.float32, (B, Hkv, S)),
            positions=positions if positions is None else _dense("source positions", positions, torch.int32, (B, Hkv, S)),
            len=lengths if lengths is None else _dense("source lengths", lengths, torch.int32, (B,)),
            next_pos=next_pos if next_pos is None else _dense("source next_pos", next_pos, torch.int32, (B,)))
        csa.csa_cache_compress(self.desc, src, stream=stream)


class SharedPrefixDecoder:
    """Decode steps of sequences that share prefixes, over a ``TokenCache``
    (csa_prefix_decode).

    Kp, Vp: [N, Hkv, Tp, D] in the cache's dtype (any strides, last index
    dense), prefix_len [N] int32 (default Tp), group_start [N + 1] int32:
    sequences group_start[n] .. group_start[n+1]-1 share prefix n (default: one
    prefix for all).  accumulate: add each step's attention weights on the own
    slots to cache.weights, the old sums times `decay` first.  rotary: turns
    the queries and new keys of ``step`` at cache.next_pos.  An inactive sequence
    (cache.next_pos negative) gets out = 0 and lse = -inf, and its sums stay."""

    def __init__(self, cache: TokenCache, *, Hq: int, Kp=None, Vp=None, prefix_len=None,
                 group_start=None, accumulate: bool = True, decay: float = 1.0,
                 scale: float | None = None, out_dtype=torch.float32, rotary: Rotary | None = None):
        B, Hkv, T, D, dt, dev = cache.B, cache.Hkv, cache.T, cache.D, cache.K.dtype, cache.K.device
        self.cache, self.Hq, self.rotary = cache, Hq, rotary
        _typed("out_dtype", out_dtype)
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        # what attend() would refuse on every call is refused here, before a step's insert
        if not (math.isfinite(scale) and scale > 0):
            _bad("scale must be finite and positive")
        if not (math.isfinite(decay) and decay >= 0):
            _bad("decay must be finite and non-negative")
        N = Tp = 0
        kw = {}
        if Kp is not None:
            N, _, Tp, _ = Kp.shape
            if N > 1 and group_start is None:
                _bad("group_start is required for more than one prefix")
            if Vp is None:
                _bad("Kp without Vp")
            kw = dict(Kp=Kp, Vp=Vp, kp_stride=_rows("Kp", Kp, dt, (N, Hkv, Tp, D)),
                      vp_stride=_rows("Vp", Vp, dt, Kp.shape))
            if prefix_len is not None:
                kw["prefix_len"] = _dense("prefix_len", prefix_len, torch.int32, (N,))
            if group_start is not None:
                kw["group_start"] = _dense("group_start", group_start, torch.int32, (N + 1,))
        for name, t in (("K", cache.K), ("V", cache.V), ("Kp", Kp), ("Vp", Vp)):
            if t is not None and t.numel() > 0:
                _wide_rows(name, t)
        self.prefix = (Kp, Vp, prefix_len, group_start)  # kept alive with the descriptor
        _same_device(dev, Kp=Kp, Vp=Vp, prefix_len=prefix_len, group_start=group_start)
        self.out = torch.empty(B, Hq, D, dtype=out_dtype, device=dev)
        self.lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
        self.q = torch.empty(B, Hq, D, dtype=dt, device=dev)  # the turned queries of step
        self.k = torch.empty(B, Hkv, D, dtype=dt, device=dev)
        with torch.cuda.device(dev):
            nbytes = csa.csa_prefix_decode_workspace_bytes(dt, B, Hq, Hkv, D, N, Tp, T, accumulate)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.desc = csa.prefix_decode_desc(
            dtype=dt, B=B, Hq=Hq, Hkv=Hkv, D=D, scale=scale,
            N=N, Tp=Tp, T=T, K=cache.K, V=cache.V, k_stride=cache.k_stride, v_stride=cache.v_stride,
            len=cache.lengths, out=self.out, out_dtype=out_dtype, lse_out=self.lse,
            weights=cache.weights if accumulate else None, decay=decay, workspace=self.workspace,
            workspace_bytes=nbytes, next_pos=cache.next_pos, **kw)

    def attend(self, q: torch.Tensor, stream=None):
        """Attention of q [B, Hq, D] over the prefixes and the cache as they
        are; returns (out, lse), this decoder's buffers."""
        _dense("q", q, self.cache.K.dtype, self.out.shape)
        return self._attend(q, stream)

    def _attend(self, q, stream):
        self.desc.q = q.data_ptr()
        csa.csa_prefix_decode(self.desc, stream=stream)
        return self.out, self.lse

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None):
        """One decode step: q [B, Hq, D] and k [B, Hkv, D] are turned to the next
        position (when there is a rotary), k and v enter the cache, and q attends.
        For serving: no gradient is kept."""
        c = self.cache
        if self.rotary is not None:
            q, k = (x.detach() if x.requires_grad else x for x in (q, k))
            self.rotary.rotate(q[:, None], k[:, None], positions=c.next_pos[:, None],
                               q_out=self.q[:, None], k_out=self.k[:, None], stream=stream)
            q, k = self.q, self.k
        # before the cache changes
        _dense("q", q, c.K.dtype, self.out.shape)
        if q.device != self.out.device or q.data_ptr() % 16:
            _bad(f"q must be on {self.out.device} and start on 16 bytes")
        c.insert(k, v, stream=stream)
        return self._attend(q, stream)
