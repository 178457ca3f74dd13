"""One attention layer's chunk-recurrent training step through the C ABI.

"Out of the Memory Barrier" (gist.science explainer, 2.A "Chunk-Recurrent Training
with Activation Recomputation"): the layer input X is processed chunk by chunk.
Forward sweep, chunk c in order: Q, K, V projected from X (optional biases), the
rotary embedding on Q and K, K/V appended to the paged pool, pages selected, the
attention forward.  Reverse sweep, chunk c from the last: Q recomputed from X, the
attention forward recomputed, the attention backward (dK/dV added into the paged
gradient pool); the chunk's keys are seen only by queries of this and later chunks,
all done by now, so its dK/dV are complete and go back through the rotary embedding
(inverse rotation) and the projections: dX, dWq, dWk, dWv and the bias gradients.

Optional parts of a layer, each off by default:
 - ``softcap``, ``slopes`` (constructor) and ``doc_start``, ``prefix_len`` (run): capped
   scores, a distance bias per head, packed documents and their bidirectional prefixes
   (oomb_score_attn_fwd/bwd, oomb_doc_spans);
 - ``pair_axis`` (constructor) with ``positions`` (run): rotary positions in several axes
   (oomb_bias_rope_axes);
 - ``w_norm`` (constructor): the norm in front of the projections, and with ``Y`` (run), the
   previous block's output, that block's own norm, gate and residual scale
   (oomb_block_norm_fwd/bwd).  Like the queries the normed input is formed again in the
   reverse sweep.

This module only orders calls; every operation is a liboomb entry point (GEMMs on
cuBLASLt through oomb_gemm, the rotation in oomb_bias_rope, the attention path).
torch provides the buffers.  Gradient GEMMs run in fp32 (the projection GEMMs in
the layer's dtype with fp32 accumulation).
"""
from __future__ import annotations

import math
from typing import List, Optional

import torch

from . import _lib as L
from .pool import PagedKVPool


def prefix_cut(doc_start, prefix_len, chunk: int, n: int):
    """Which documents' prefixes a layer step that goes ``chunk`` by chunk over ``n`` tokens cannot show to
    all of their rows: those that go past the end of the chunk in which their document starts (a
    chunk's keys are not there yet when the one before attends).  Bool [n_docs], where doc_start is."""
    first, last = doc_start[:-1].clamp(0, n), doc_start[1:].clamp(0, n)
    end = torch.minimum(doc_start[:-1] + torch.minimum(prefix_len, doc_start[1:] - doc_start[:-1]), last)
    return (end > first) & ((end - 1) // chunk > first // chunk)


def chunk_gradient(d_o, o):
    """A chunk's dO, whose memory the kernels read as that of ``o``: of its dtype and device, as many elements,
    contiguous.  Anything else is refused."""
    if not isinstance(d_o, torch.Tensor) or d_o.dtype is not o.dtype:
        raise TypeError(f"LayerStep: dO has to be {o.dtype}, not {getattr(d_o, 'dtype', type(d_o).__name__)}")
    if d_o.device != o.device:
        raise ValueError(f"LayerStep: dO is on {d_o.device}, not on {o.device}")
    if d_o.numel() != o.numel():
        raise ValueError(f"LayerStep: dO of a chunk has shape {tuple(d_o.shape)}, needs {tuple(o.shape)}")
    if not d_o.is_contiguous():
        raise ValueError("LayerStep: dO is not contiguous")
    return d_o


class LayerStep:
    """Weights Wq [Dm, Hq*d], Wk and Wv [Dm, Hkv*d] (the pool's dtype, device), biases
    fp32 [H*d] or None.  Selection: top-K (``top_k``, ``n_sink``) or a local window
    (``window`` >= 0).

    ``softcap`` (0: none) and ``slopes`` (fp32 [Hq]): the scores' cap and distance bias.
    ``pair_axis`` (d/2 axis numbers): rotary positions in several axes, given to ``run``;
    ``own_ladder``: each axis has a frequency ladder of its own.
    ``w_norm`` (fp32 [Dm]): u = norm(x) in front of the projections, x the residual stream;
    ``w_post`` (fp32 [Dm] or None), ``gate`` (fp32 [Dm] or None) and ``res_scale``: with the
    previous block's output Y, x = X + res_scale * gate * norm(Y; w_post)."""

    def __init__(self, pool: PagedKVPool, Wq, Wk, Wv, bq=None, bk=None, bv=None, chunk: int = 4096,
                 theta: float = 1e6, top_k: int = -1, n_sink: int = 1, window: int = -1,
                 gemm_workspace_bytes: int = 32 << 20, softcap: float = 0.0, slopes=None, pair_axis=None,
                 own_ladder: bool = False, w_norm=None, w_post=None, gate=None, res_scale: float = 1.0,
                 eps: float = 1e-6):
        if w_norm is None and (w_post is not None or gate is not None):
            raise ValueError("LayerStep: w_post and gate belong to the norm in front of the layer (w_norm)")
        self.softcap, self.slopes = softcap, slopes
        self.pair_axis, self.own_ladder = pair_axis, own_ladder
        self.w_norm, self.w_post, self.gate, self.res_scale, self.eps = w_norm, w_post, gate, res_scale, eps
        self.pool, self.chunk, self.theta = pool, chunk, theta
        self.top_k, self.n_sink, self.window = top_k, n_sink, window
        self.Hq, self.Hkv, self.d, self.P = pool.Hq, pool.Hkv, pool.d, pool.P
        self.dev = pool.device
        self.W = {"q": Wq, "k": Wk, "v": Wv}
        self.b = {"q": bq, "k": bk, "v": bv}
        self.Dm = Wq.shape[0]
        self.scale = 1.0 / math.sqrt(self.d)
        self.ws = torch.empty(gemm_workspace_bytes, dtype=torch.uint8, device=self.dev)
        # fp32 copies of the weights for the gradient GEMMs (a cast through oomb_bias_rope)
        self.W32 = {}
        for key, w in self.W.items():
            w32 = torch.empty(w.shape, dtype=torch.float32, device=self.dev)
            L.oomb_bias_rope(w, None, w32, w.numel() // (w.shape[0] * 2), 0, 0.0, 0)
            self.W32[key] = w32

    # ------------------------------------------------------------------ pieces
    def _rotate(self, x_in, bias, x_out, H: int, pos0: int, mode: int):
        """oomb_bias_rope at positions pos0.., or at the run's positions of those tokens."""
        if self.pair_axis is None or mode == 0:
            L.oomb_bias_rope(x_in, bias, x_out, H, pos0, self.theta, mode)
        else:
            pos = self._positions[:, pos0:pos0 + x_in.shape[0]].contiguous()
            L.oomb_bias_rope_axes(x_in, bias, x_out, H, pos, self.pair_axis, self.theta, mode,
                                  own_ladder=self.own_ladder)

    def _project(self, x, key: int, H: int, pos0: int, rotate: bool):
        """[n, H, d] in the pool's dtype: rotation(pos0..) (x W + b)."""
        n = x.shape[0]
        acc = torch.empty((n, H * self.d), dtype=torch.float32, device=self.dev)
        L.oomb_gemm(x, self.W[key], acc, workspace=self.ws)
        out = torch.empty((n, H, self.d), dtype=self.pool.dtype, device=self.dev)
        self._rotate(acc, self.b[key], out, H, pos0, 1 if rotate else 0)
        return out

    def _input(self, x, y, keep=None):
        """The projections' input: x, or its norm.  ``keep`` [n, Dm] gets the residual stream."""
        if self.w_norm is None:
            return x, None
        n = x.shape[0]
        u = torch.empty_like(x)
        if keep is None and y is not None:
            keep = torch.empty_like(x)
        rstd = [torch.empty(n, dtype=torch.float32, device=self.dev) if w is not None else None
                for w in (self.w_norm, None if y is None else self.w_post)]
        L.oomb_block_norm_fwd(x, y, keep, u, w_pre=self.w_norm, w_post=None if y is None else self.w_post,
                              gate=None if y is None else self.gate, res_scale=self.res_scale, eps=self.eps,
                              rstd_pre=rstd[0], rstd_post=rstd[1])
        return u, rstd

    def _attend(self, q, s: int, sel, o, lse):
        """The chunk's attention forward, with the scores this layer uses."""
        h = self.pool.handle
        if not self._scores:
            L.oomb_chunk_attn_fwd(h, q, s, sel[0], sel[1], self.scale, o, lse)
            return
        L.oomb_score_attn_fwd(h, q, s, sel[0], sel[1], self.scale, o, lse, self._ws_fwd, **self._mod(s, q.shape[0]))

    def _attend_bwd(self, q, o, d_o, lse, s: int, sel, dq, ws):
        h = self.pool.handle
        if not self._scores:
            L.oomb_chunk_attn_bwd(h, q, o, d_o, lse, s, sel[0], sel[1], self.scale, dq, ws)
            return
        L.oomb_score_attn_bwd(h, q, o, d_o, lse, s, sel[0], sel[1], self.scale, dq, ws, **self._mod(s, q.shape[0]))

    def _mod(self, s: int, n: int) -> dict:
        """The score arguments of the chunk at s (its key ranges, where there are documents)."""
        mod = dict(softcap=self.softcap, slopes=self.slopes)
        if self._docs is not None:
            begin, end = (torch.empty(n, dtype=torch.int64, device=self.dev) for _ in range(2))
            L.oomb_doc_spans(self._docs[0], s, begin, end, prefix_len=self._docs[1])
            mod.update(key_begin=begin, key_end=end)
        return mod

    def _select(self, q, start: int, sel, cnt, ws_sel):
        h = self.pool.handle
        if self.window >= 0:
            L.oomb_window_select(h, start, q.shape[0], self.window, self.n_sink, sel, cnt)
        else:
            L.oomb_page_select(h, q, start, self.top_k, self.n_sink, sel, cnt, ws_sel)

    def max_sel(self) -> int:
        own = -(-self.chunk // self.P)
        if self.window >= 0:
            return self.n_sink + self.window + own
        if self.top_k < 0:
            return self.pool.max_logical
        return self.n_sink + self.top_k + own

    # ------------------------------------------------------------------ the step
    def run(self, X, dO, sel_override: Optional[List] = None, Y=None, dX_out=None, positions=None, doc_start=None,
            prefix_len=None) -> dict:
        """X [N, Dm] (pool dtype, device), dO [N, Hq, d] (pool dtype, device), or a function that
        forms a chunk's dO when the reverse sweep has recomputed its output: dO(first token, o [n, Hq, d])
        (ModelEnds.behind: the loss of the chunk).
        ``sel_override[c]``: (sel, count) device tensors fed to chunk c's attention
        instead of the library's own selection (which is still computed and returned).
        Returns O (per chunk), sel (the library's selections, per chunk), dX, dWq, dWk,
        dWv, dbq, dbk, dbv (fp32; the bias gradients are zero where there is no bias).

        ``positions`` int64 [n_axes, N] with ``pair_axis``.  ``doc_start`` int64 [n_docs + 1]
        and optionally ``prefix_len`` int64 [n_docs]: packed documents; a row sees its own
        document only, and keys of this and earlier chunks (so a prefix that is to be seen by
        all of its rows has to end with its chunk; ``prefix_cut`` of the result, bool [n_docs], says
        whose does not).  The library's top-K selection and its sink
        pages do not know the documents: with ``doc_start`` every page is kept (``top_k`` = -1), a
        window goes without sinks, or the pages are given.  With ``w_norm``: ``Y`` [N, Dm], the
        previous block's output, and ``dX_out`` [N, Dm], the gradient that reaches the residual
        stream behind this layer; also returned are X_out (the residual stream), dY, and fp32
        dw_norm, dw_post, dgate (those that exist); dX and dY are then in the pool's dtype.
        Errors that kernels met are told by oomb_check (the pool) and, with ``w_norm``,
        oomb_block_norm_check."""
        if (positions is None) != (self.pair_axis is None):
            raise ValueError("LayerStep: positions and pair_axis come together")
        if self.w_norm is None and (Y is not None or dX_out is not None):
            raise ValueError("LayerStep: Y and dX_out need the norm in front of the layer (w_norm)")
        if Y is None and (self.w_post is not None or self.gate is not None):
            raise ValueError("LayerStep: w_post and gate act on Y")
        if prefix_len is not None and doc_start is None:
            raise ValueError("LayerStep: prefix_len needs doc_start")
        if doc_start is not None and sel_override is None and (self.n_sink > 0 if self.window >= 0 else self.top_k >= 0):
            raise ValueError("LayerStep: the top-K selection and the sink pages do not know documents and would pick "
                             "pages that are masked; keep every page (top_k = -1), take a window without sinks, or "
                             "give the pages (sel_override)")
        self._positions = positions
        self._docs = None if doc_start is None else (doc_start, prefix_len)
        self._scores = self.softcap != 0.0 or self.slopes is not None or self._docs is not None
        try:
            out = self._run(X, dO, sel_override, Y, dX_out)
        finally:  # nothing of a call is kept for the next
            self._positions = self._docs = self._ws_fwd = None
        if prefix_len is not None:
            out["prefix_cut"] = prefix_cut(doc_start, prefix_len, self.chunk, X.shape[0])
        return out

    def _run(self, X, dO, sel_override, Y, dX_out) -> dict:
        pool, h, dev = self.pool, self.pool.handle, self.dev
        N, Dm, Hq, Hkv, d = X.shape[0], self.Dm, self.Hq, self.Hkv, self.d
        if self._scores:
            self._ws_fwd = pool.workspace(L.OOMB_OP_SCORE_FWD, self.chunk)
        starts = list(range(0, N, self.chunk))
        L.oomb_pool_reset(h)
        max_sel = self.max_sel()
        ws_sel = pool.workspace(L.OOMB_OP_SELECT, self.chunk)
        ws_bwd = pool.workspace(L.OOMB_OP_SCORE_BWD if self._scores else L.OOMB_OP_BWD, self.chunk)
        out = {"O": [], "sel": []}
        norm = self.w_norm is not None
        cut = lambda t, s, n: None if t is None else t[s:s + n]  # noqa: E731
        if norm:
            out["X_out"] = torch.empty_like(X) if Y is not None else X
        att = []  # the selection each chunk's attention used
        for ci, s in enumerate(starts):
            n = min(self.chunk, N - s)
            x, _ = self._input(X[s:s + n], cut(Y, s, n), cut(out["X_out"], s, n) if Y is not None else None)
            q = self._project(x, "q", Hq, s, True)
            k = self._project(x, "k", Hkv, s, True)
            v = self._project(x, "v", Hkv, s, False)
            L.oomb_kv_append(h, k, v, s)
            sel = torch.full((Hkv, max_sel), -1, dtype=torch.int32, device=dev)
            cnt = torch.zeros(Hkv, dtype=torch.int32, device=dev)
            self._select(q, s, sel, cnt, ws_sel)
            out["sel"].append((sel, cnt))
            a_sel = sel_override[ci] if sel_override is not None else (sel, cnt)
            att.append(a_sel)
            o = torch.empty_like(q)
            lse = torch.empty((Hq, n), dtype=torch.float32, device=dev)
            self._attend(q, s, a_sel, o, lse)
            out["O"].append(o)
        f32 = torch.float32
        dX = torch.empty((N, Dm), dtype=f32, device=dev)
        if norm:
            out["dX"] = torch.empty_like(X)
            out["dY"] = None if Y is None else torch.empty_like(Y)
            dp = {key: None if w is None or (Y is None and key != "dw_norm") else torch.zeros_like(w)
                  for key, w in (("dw_norm", self.w_norm), ("dw_post", self.w_post), ("dgate", self.gate))}
            ws_norm = torch.empty(L.oomb_block_norm_workspace(self.chunk, Dm), dtype=torch.uint8, device=dev)
        dW = {key: torch.zeros(self.W[key].shape, dtype=f32, device=dev) for key in "qkv"}
        db = {key: torch.zeros((1, self.W[key].shape[1]), dtype=f32, device=dev) for key in "qkv"}
        ones = torch.ones((1, self.chunk), dtype=f32, device=dev)
        for ci in range(len(starts) - 1, -1, -1):
            s = starts[ci]
            n = min(self.chunk, N - s)
            x, rstd = self._input(X[s:s + n], cut(Y, s, n))
            q = self._project(x, "q", Hq, s, True)  # recomputed (explainer 2.A)
            o = torch.empty_like(q)
            lse = torch.empty((Hq, n), dtype=torch.float32, device=dev)
            a_sel = att[ci]
            self._attend(q, s, a_sel, o, lse)
            dq = torch.empty_like(q)
            d_o = chunk_gradient(dO(s, o) if callable(dO) else dO[s:s + n], o)
            self._attend_bwd(q, o, d_o, lse, s, a_sel, dq, ws_bwd)
            # the chunk's own dK/dV are complete: back through the rotation and projections
            g = {"q": torch.empty((n, Hq * d), dtype=f32, device=dev),
                 "k": torch.empty((n, Hkv * d), dtype=f32, device=dev),
                 "v": torch.empty((n, Hkv * d), dtype=f32, device=dev)}
            L.oomb_grad_gather(h, s, g["k"].view(n, Hkv, d), g["v"].view(n, Hkv, d))
            self._rotate(dq, None, g["q"], Hq, s, 2)
            self._rotate(g["k"], None, g["k"], Hkv, s, 2)
            x32 = torch.empty((n, Dm), dtype=f32, device=dev)
            L.oomb_bias_rope(x, None, x32, Dm // 2, 0, 0.0, 0)  # cast
            first = True
            for key in "qkv":
                L.oomb_gemm(x32, g[key], dW[key], trans_a=True, beta=1.0, workspace=self.ws)
                L.oomb_gemm(ones[:, :n], g[key], db[key], beta=1.0, workspace=self.ws)
                L.oomb_gemm(g[key], self.W32[key], dX[s:s + n], trans_b=True, beta=0.0 if first else 1.0,
                            workspace=self.ws)
                first = False
            if norm:
                # the norm's backward reads its rows in the residual stream's type, so the gradient of the
                # normed input, summed in fp32 over the three projections, is rounded to it once here
                du = dX[s:s + n]
                if pool.dtype != f32:
                    du = torch.empty((n, Dm), dtype=pool.dtype, device=dev)
                    L.oomb_bias_rope(dX[s:s + n], None, du, Dm // 2, 0, 0.0, 0)  # cast
                block = Y is not None
                L.oomb_block_norm_bwd(X[s:s + n], cut(Y, s, n), out["dX"][s:s + n], cut(out["dY"], s, n), du=du,
                                      dx_out=cut(dX_out, s, n), rstd_pre=rstd[0], rstd_post=rstd[1],
                                      w_pre=self.w_norm, w_post=self.w_post if block else None,
                                      gate=self.gate if block else None, dw_pre=dp["dw_norm"], dw_post=dp["dw_post"],
                                      dgate=dp["dgate"], res_scale=self.res_scale, accumulate=True, workspace=ws_norm)
        if norm:
            dX = out["dX"]
            out.update({key: g for key, g in dp.items() if g is not None})
        out.update(dX=dX, dWq=dW["q"], dWk=dW["k"], dWv=dW["v"], dbq=db["q"][0], dbk=db["k"][0], dbv=db["v"][0])
        return out
