"""Operators of the layer step, measured: plain forms, the framework's calls, exact values.

Three families, the ones that stand around the paged chunk attention of a training
layer and that the layer step calls:

attn   chunk attention over the paged cache whose scores are capped by a tanh, get a
       bias that falls with distance, and are masked by document and by prefix;
       forward, and forward + backward (dQ, and dK/dV from the paged pools)
norm   the norms before and after a block fused with the block's gate and residual
       scale; forward, and forward + backward
rope   rotary positions with several axes (time, height, width), forward and inverse

A case is a dict of plain values; ``draw`` gives more of the same ranges.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------- cases
def _attn(name, train, dtype, Hq, Hkv, d, P, n_tokens, n_q, top_k, cap, bias, docs, prefix):
    """docs: mean document length (0: one document); top_k: history pages per KV head
    besides the first one (-1: every page); the chunk is the last n_q of n_tokens."""
    return {"name": name, "kind": "attn", "train": train, "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "d": d, "P": P,
            "n_tokens": n_tokens, "n_q": n_q, "top_k": top_k, "cap": cap, "bias": bias, "docs": docs,
            "prefix": prefix}


def _norm(name, train, dtype, n, D, gate, post, block=True):
    return {"name": name, "kind": "norm", "train": train, "dtype": dtype, "n": n, "D": D, "gate": gate,
            "post": post, "block": block}


def _rope(name, n, H, d, in_dtype, out_dtype, axes, layout, ladder, mode, bias):
    return {"name": name, "kind": "rope", "n": n, "H": H, "d": d, "in_dtype": in_dtype, "out_dtype": out_dtype,
            "axes": axes, "layout": layout, "ladder": ladder, "mode": mode, "bias": bias}


def listed():
    return [
        # one new token behind a 128K-token cache, every page read: the serving call, where
        # the long axis has to be split for one row to use the whole GPU
        _attn("attn_token_128k", False, "bf16", 28, 4, 128, 128, 131072, 1, -1, 30.0, True, 0, False),
        # a short tail of new tokens (a last chunk) over a page selection: latency
        _attn("attn_tail_sel", False, "bf16", 28, 4, 128, 128, 32768 + 17, 17, 64, 50.0, False, 0, False),
        # one chunk of the 128K workload with capped scores
        _attn("attn_chunk_cap", False, "bf16", 28, 4, 128, 128, 131072, 4096, 64, 50.0, False, 0, False),
        # packed documents with a bidirectional prefix each, distance bias, whole cache kept
        _attn("attn_docs_prefix", False, "bf16", 28, 4, 128, 128, 65536, 8192, -1, 0.0, True, 12000, True),
        # training on one 8K chunk of the long workloads: top-128 pages, capped scores
        _attn("attn_train_cap_8k", True, "bf16", 28, 4, 128, 128, 65536, 8192, 128, 50.0, False, 0, False),
        # training on packed documents: ragged chunk, everything on at once
        _attn("attn_train_docs", True, "bf16", 28, 4, 128, 128, 12001, 4001, -1, 30.0, True, 1500, True),
        # the fp32 configuration (2 query heads, 1 KV head, 64 wide, pages of 64)
        _attn("attn_train_fp32", True, "fp32", 2, 1, 64, 64, 4096, 1024, -1, 20.0, True, 1000, False),
        # one token through a sandwich of norms at the stack's model width: launch latency
        _norm("norm_token", False, "bf16", 1, 3584, "channel", True),
        # one 8K chunk at that width, forward and backward, weight gradients included
        _norm("norm_train_8k", True, "bf16", 8192, 3584, "channel", True),
        # fp32, odd width, a gate for each token and channel
        _norm("norm_train_odd", True, "fp32", 1001, 1537, "token", True),
        # queries of an 8K chunk of video, positions in three axes taken in turn, from the
        # projection's fp32 output with its bias to the attention's bf16
        _rope("rope_video_q", 8192, 28, 128, "fp32", "bf16", 3, "turns", False, 1, True),
        # gradients of an image's keys turned back: two axes with a frequency ladder each
        _rope("rope_image_grad", 1001, 16, 80, "bf16", "fp32", 2, "blocks", True, 2, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "norm", "rope"])
    if kind == "attn":
        train = rng.random() < 0.5
        tc = rng.random() < 0.75
        if tc:
            dtype, (Hq, Hkv), d, P = "bf16", rng.choice([(28, 4), (16, 2), (8, 8), (12, 4)]), 128, 128
            n_q = _log_int(rng, 1, 8192)
            n_tokens = min(65536, n_q + _log_int(rng, 64, 57000))
        else:
            dtype, d, P = rng.choice([("fp32", 64, 64), ("fp32", 128, 16), ("bf16", 64, 64), ("bf16", 96, 32)])
            Hq, Hkv = rng.choice([(2, 1), (4, 4), (6, 2)])
            n_q = _log_int(rng, 1, 1024)
            n_tokens = n_q + _log_int(rng, 16, 3000)
        docs = rng.choice([0, 0, _log_int(rng, 100, 20000)])
        top_k = rng.choice([-1, _log_int(rng, 1, 128)]) if not docs else -1
        cap = rng.choice([0.0, 20.0, 30.0, 50.0])
        bias = rng.random() < 0.5 or (cap == 0.0 and not docs)
        return _attn("", train, dtype, Hq, Hkv, d, P, n_tokens, n_q, top_k, cap, bias, docs,
                     bool(docs) and rng.random() < 0.5)
    if kind == "norm":
        D = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        n = _log_int(rng, 1, min(8192, 8192 * 3584 // D))
        return _norm("", rng.random() < 0.6, rng.choice(["bf16", "bf16", "fp32"]), n, D,
                     rng.choice(["none", "channel", "token"]), rng.random() < 0.7)
    d = rng.choice([64, 80, 96, 128, 24, 72])
    H = rng.choice([1, 4, 7, 16, 28])
    n = _log_int(rng, 1, min(8192, 8192 * 28 * 128 // (H * d)))
    mode = rng.choice([1, 1, 2])
    return _rope("", n, H, d, rng.choice(["fp32", "bf16"]), rng.choice(["fp32", "bf16"]), rng.choice([1, 2, 3, 4]),
                 rng.choice(["turns", "blocks"]), rng.random() < 0.5, mode, mode == 1 and rng.random() < 0.5)


# ------------------------------------------------------- shapes told by the case
def _tdt(s):
    return torch.float32 if s == "fp32" else torch.bfloat16


def _doc_starts(case):
    """Document boundaries [0, ..., n_tokens] and prefix lengths, from the case alone."""
    N = case["n_tokens"]
    if not case["docs"]:
        return None, None
    r = random.Random("docs %d %d" % (N, case["docs"]))
    cuts = [0]
    while cuts[-1] < N:
        cuts.append(min(N, cuts[-1] + max(1, int(case["docs"] * (0.4 + 1.2 * r.random())))))
    pre = [int((b - a) * 0.3 * r.random()) for a, b in zip(cuts[:-1], cuts[1:])] if case["prefix"] else None
    return cuts, pre


def _spans(case):
    """Visible key range [begin, end) of each query row, as two int64 numpy arrays."""
    q0 = case["n_tokens"] - case["n_q"]
    pos = np.arange(q0, case["n_tokens"], dtype=np.int64)
    cuts, pre = _doc_starts(case)
    if cuts is None:
        return np.zeros_like(pos), pos + 1
    which = np.searchsorted(np.asarray(cuts), pos, side="right") - 1
    begin = np.asarray(cuts, dtype=np.int64)[which]
    end = pos + 1
    if pre is not None:
        end = np.maximum(end, begin + np.asarray(pre, dtype=np.int64)[which])
    return begin, end


def _page_counts(case):
    """Pages of the cache, first page of the chunk, history pages kept for each KV head."""
    P, N = case["P"], case["n_tokens"]
    n_pages, own0 = -(-N // P), (N - case["n_q"]) // P
    kept = own0 if case["top_k"] < 0 else min(own0, 1 + case["top_k"])
    return n_pages, own0, kept


def _pair_axis(case):
    half, A = case["d"] // 2, case["axes"]
    if case["layout"] == "turns":
        return [j % A for j in range(half)]
    return [min(A - 1, j * A // half) for j in range(half)]


def _visible_pairs(case):
    """(query row, key) pairs seen by one query head (expected value under a selection)."""
    begin, end = _spans(case)
    n_pages, own0, kept = _page_counts(case)
    o = own0 * case["P"]
    hist = np.clip(np.minimum(end, o) - np.minimum(begin, o), 0, None).sum()
    mine = np.clip(end - np.maximum(begin, o), 0, None).sum()
    frac = kept / own0 if own0 else 0.0
    return float(hist) * frac + float(mine)


def work(case):
    if case["kind"] == "attn":
        es = 4 if case["dtype"] == "fp32" else 2
        Hq, Hkv, d, n_q, P = case["Hq"], case["Hkv"], case["d"], case["n_q"], case["P"]
        begin, end = _spans(case)
        n_pages, own0, kept = _page_counts(case)
        lo = int(begin.min())
        keys = max(0, own0 * P - lo) * (kept / own0 if own0 else 0.0) + case["n_tokens"] - max(lo, own0 * P)
        pairs = _visible_pairs(case) * Hq
        q_bytes, kv_bytes = n_q * Hq * d * es, keys * Hkv * d * 2 * es
        if not case["train"]:
            return {"bytes": 2 * q_bytes + kv_bytes + 4 * n_q * Hq, "flops": 4.0 * d * pairs}
        # Q, dO in, O, dQ out; K, V in; the two gradients of every page out
        return {"bytes": 4 * q_bytes + kv_bytes + 4 * n_q * Hq + 2 * es * n_pages * P * Hkv * d,
                "flops": 14.0 * d * pairs}
    if case["kind"] == "norm":
        n, D, es = case["n"], case["D"], (4 if case["dtype"] == "fp32" else 2)
        tok = case["gate"] == "token"
        if not case["train"]:
            return {"bytes": n * D * es * (4 + tok) + 12 * D, "flops": 10.0 * n * D}
        # x, y, (gate), du, dx' in; x', u, dx, dy, (dgate) out
        return {"bytes": n * D * es * (8 + 2 * tok) + 24 * D, "flops": 40.0 * n * D}
    es = (4 if case["in_dtype"] == "fp32" else 2) + (4 if case["out_dtype"] == "fp32" else 2)
    return {"bytes": case["n"] * case["H"] * case["d"] * es + 8 * case["axes"] * case["n"],
            "flops": 4.0 * case["n"] * case["H"] * case["d"]}


# --------------------------------------------------------------------- inputs
def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 9973 + 17)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    st = {"case": case}
    if case["kind"] == "attn":
        N, n_q, Hq, Hkv, d, P = (case[k] for k in ("n_tokens", "n_q", "Hq", "Hkv", "d", "P"))
        dt = _tdt(case["dtype"])
        # queries and keys of trained layers score well above unit variance
        st["q"] = (rn(n_q, Hq, d) * 2.0).to(dt)
        st["k"] = rn(N, Hkv, d).to(dt)
        st["v"] = rn(N, Hkv, d).to(dt)
        if case["train"]:
            st["do"] = rn(n_q, Hq, d).to(dt)
        st["scale"] = 1.0 / math.sqrt(d)
        # distance slopes: a geometric sequence over the heads
        st["slopes"] = (2.0 ** (-8.0 * (torch.arange(Hq, device=DEV, dtype=torch.float32) + 1) / Hq)
                        if case["bias"] else None)
        cuts, pre = _doc_starts(case)
        st["doc_start"] = None if cuts is None else torch.tensor(cuts, dtype=torch.int64, device=DEV)
        st["prefix_len"] = None if pre is None else torch.tensor(pre, dtype=torch.int64, device=DEV)
        n_pages, own0, kept = _page_counts(case)
        gc = torch.Generator()
        gc.manual_seed(int(seed) * 31 + 5)
        rows = []
        for _ in range(Hkv):  # first page, `kept - 1` retrieved ones, the chunk's own; ascending
            hist = (torch.cat([torch.zeros(1, dtype=torch.long),
                               1 + torch.randperm(own0 - 1, generator=gc)[:kept - 1].sort().values])
                    if kept > 0 else torch.zeros(0, dtype=torch.long))
            rows.append(torch.cat([hist, torch.arange(own0, n_pages)]))
        sel = torch.stack(rows)
        st["sel_cpu"] = sel
        st["sel"] = sel.to(torch.int32).to(DEV)
        st["sel_count"] = torch.full((Hkv,), sel.shape[1], dtype=torch.int32, device=DEV)
        st["order"] = torch.randperm(n_pages, generator=gc)  # physical page of each logical one
    elif case["kind"] == "norm":
        n, D, dt = case["n"], case["D"], _tdt(case["dtype"])
        wide = 1.0 + 8.0 * (torch.rand(D, generator=g, device=DEV) > 0.99).float()  # a few loud channels
        st["x"] = (rn(n, D) * 2.0 * wide).to(dt)
        st["y"] = (rn(n, D) * 0.7).to(dt)
        st["w_pre"] = 1.0 + 0.2 * rn(D)
        st["w_post"] = 1.0 + 0.2 * rn(D) if case["post"] else None
        st["gate"] = {"none": None, "channel": 0.5 + 0.1 * rn(D),
                      "token": torch.sigmoid(rn(n, D)).to(dt)}[case["gate"]]
        st["res_scale"], st["eps"] = 0.7, 1e-6
        if case["train"]:
            st["du"], st["dx_out"] = rn(n, D).to(dt), rn(n, D).to(dt)
    else:
        n, H, d, A = case["n"], case["H"], case["d"], case["axes"]
        st["x"] = rn(n, H, d).to(_tdt(case["in_dtype"]))
        st["bias"] = rn(H * d) if case["bias"] else None
        # frames of a patch grid deep inside a long video: time far out, height and width small
        t = torch.arange(n, device=DEV)
        pos = [4_000_000 + t // 64, (t // 8) % 8 + int(seed) % 5, t % 8, t]
        st["positions"] = torch.stack(pos[:A]).to(torch.int64).contiguous()
        st["pair_axis"], st["theta"] = _pair_axis(case), 1e6
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own:
        return st
    import paged_sparse_attention_gb300 as L
    from paged_sparse_attention_gb300.pool import PagedKVPool

    if case["kind"] == "attn":
        n_pages = st["order"].numel()
        pool = PagedKVPool(case["Hq"], case["Hkv"], case["d"], case["P"], n_pages, n_pages, _tdt(case["dtype"]),
                           torch.device(DEV, torch.cuda.current_device()), page_order=st["order"])
        L.oomb_kv_append(pool.handle, st["k"], st["v"], 0)
        st["pool"] = pool
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(case["Hq"], case["n_q"], dtype=torch.float32, device=DEV)
        st["ws_fwd"] = pool.workspace(L.OOMB_OP_SCORE_FWD, case["n_q"])
        if st["doc_start"] is not None:
            st["begin"] = torch.empty(case["n_q"], dtype=torch.int64, device=DEV)
            st["end"] = torch.empty(case["n_q"], dtype=torch.int64, device=DEV)
        else:
            st["begin"] = st["end"] = None
        if case["train"]:
            st["dq"] = torch.empty_like(st["q"])
            st["ws_bwd"] = pool.workspace(L.OOMB_OP_SCORE_BWD, case["n_q"])
    elif case["kind"] == "norm":
        n, D = st["x"].shape
        st["x_out"], st["u"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["rstd_pre"] = torch.empty(n, dtype=torch.float32, device=DEV)
        st["rstd_post"] = torch.empty(n, dtype=torch.float32, device=DEV) if case["post"] else None
        if case["train"]:
            st["dx"], st["dy"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
            st["dw_pre"] = torch.empty(D, dtype=torch.float32, device=DEV)
            st["dw_post"] = torch.empty(D, dtype=torch.float32, device=DEV) if case["post"] else None
            st["dgate"] = None if st["gate"] is None else torch.empty_like(st["gate"])
            st["ws"] = torch.empty(L.oomb_block_norm_workspace(n, D), dtype=torch.uint8, device=DEV)
    else:
        st["out"] = torch.empty(st["x"].shape, dtype=_tdt(case["out_dtype"]), device=DEV)
    return st


# ------------------------------------------------------------- the framework
def _run_own(st):
    import paged_sparse_attention_gb300 as L

    case = st["case"]
    if case["kind"] == "attn":
        pool, h = st["pool"], st["pool"].handle
        q0 = case["n_tokens"] - case["n_q"]
        if st["doc_start"] is not None:
            L.oomb_doc_spans(st["doc_start"], q0, st["begin"], st["end"], prefix_len=st["prefix_len"])
        mod = dict(softcap=case["cap"], slopes=st["slopes"], key_begin=st["begin"], key_end=st["end"])
        L.oomb_score_attn_fwd(h, st["q"], q0, st["sel"], st["sel_count"], st["scale"], st["o"], st["lse"],
                              st["ws_fwd"], **mod)
        if not case["train"]:
            return st["o"], st["lse"]
        pool.dk_pool.zero_()  # a step starts from empty gradient pools
        pool.dv_pool.zero_()
        L.oomb_score_attn_bwd(h, st["q"], st["o"], st["do"], st["lse"], q0, st["sel"], st["sel_count"], st["scale"],
                              st["dq"], st["ws_bwd"], **mod)
        dt = _tdt(case["dtype"])  # the fp32 pools' gradients in the type of K and V
        return st["o"], st["lse"], st["dq"], pool.dk_pool.to(dt), pool.dv_pool.to(dt)
    if case["kind"] == "norm":
        par = dict(w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"], res_scale=st["res_scale"])
        L.oomb_block_norm_fwd(st["x"], st["y"], st["x_out"], st["u"], eps=st["eps"], rstd_pre=st["rstd_pre"],
                              rstd_post=st["rstd_post"], **par)
        if not case["train"]:
            return st["x_out"], st["u"]
        L.oomb_block_norm_bwd(st["x"], st["y"], st["dx"], st["dy"], du=st["du"], dx_out=st["dx_out"],
                              rstd_pre=st["rstd_pre"], rstd_post=st["rstd_post"], dw_pre=st["dw_pre"],
                              dw_post=st["dw_post"], dgate=st["dgate"], workspace=st["ws"], **par)
        out = [st["x_out"], st["u"], st["dx"], st["dy"], st["dw_pre"]]
        return out + [t for t in (st["dw_post"], st["dgate"]) if t is not None]
    L.oomb_bias_rope_axes(st["x"], st["bias"], st["out"], case["H"], st["positions"], st["pair_axis"], st["theta"],
                          case["mode"], own_ladder=case["ladder"])
    return st["out"]


# ---------------------------------------------------------------- plain forms
def _plain_attn(st):
    case = st["case"]
    Hq, Hkv, d, P, N, n_q = (case[k] for k in ("Hq", "Hkv", "d", "P", "n_tokens", "n_q"))
    G, scale, cap, q0 = Hq // Hkv, st["scale"], case["cap"], N - n_q
    pos = torch.arange(q0, N, device=DEV)
    begin, end = torch.zeros_like(pos), pos + 1
    if st["doc_start"] is not None:
        doc = torch.searchsorted(st["doc_start"], pos, right=True) - 1
        begin = st["doc_start"][doc]
        if st["prefix_len"] is not None:
            end = torch.maximum(end, begin + st["prefix_len"][doc])
    o = torch.empty(n_q, Hq, d, device=DEV)
    lse = torch.empty(Hq, n_q, device=DEV)
    if case["train"]:
        dq = torch.empty(n_q, Hq, d, device=DEV)
        n_pages = st["order"].numel()
        dk = torch.zeros(n_pages * P, Hkv, d, device=DEV)
        dv = torch.zeros(n_pages * P, Hkv, d, device=DEV)
    lo = begin.min()
    for h in range(Hkv):
        tok = (st["sel"][h].long()[:, None] * P + torch.arange(P, device=DEV)).reshape(-1)
        tok = tok[(tok < N) & (tok >= lo)]
        k, v = st["k"][tok, h].float(), st["v"][tok, h].float()
        hidden = (tok[None, :] < begin[:, None]) | (tok[None, :] >= end[:, None])
        dist = (pos[:, None] - tok[None, :]).abs().float() if case["bias"] else None
        dk_h = dv_h = 0.0
        for hq in range(h * G, (h + 1) * G):
            q = st["q"][:, hq].float()
            s = (q @ k.T) * scale
            if cap > 0:
                t = torch.tanh(s / cap)
                s = t * cap
            if dist is not None:
                s = s - st["slopes"][hq] * dist
            s = s.masked_fill(hidden, float("-inf"))
            m = s.max(dim=1, keepdim=True).values
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            den = p.sum(dim=1, keepdim=True)
            p = p / torch.where(den > 0, den, torch.ones_like(den))
            lse[hq] = (m + torch.log(den))[:, 0]
            o_h = p @ v
            o[:, hq] = o_h
            if case["train"]:
                do = st["do"][:, hq].float()
                ds = p * (do @ v.T - (do * o_h).sum(dim=1, keepdim=True))
                if cap > 0:
                    ds = ds * (1.0 - t * t)
                dq[:, hq] = (ds @ k) * scale
                dk_h = dk_h + (ds.T @ q) * scale
                dv_h = dv_h + p.T @ do
        if case["train"]:
            dk[tok, h] = dk_h
            dv[tok, h] = dv_h
    dt = _tdt(case["dtype"])
    if not case["train"]:
        return o.to(dt), lse
    order = st["order"].to(DEV)
    pk = torch.empty(n_pages, Hkv, P, d, device=DEV)
    pv = torch.empty(n_pages, Hkv, P, d, device=DEV)
    pk[order] = dk.view(n_pages, P, Hkv, d).transpose(1, 2)
    pv[order] = dv.view(n_pages, P, Hkv, d).transpose(1, 2)
    return o.to(dt), lse, dq.to(dt), pk.to(dt), pv.to(dt)


def _plain_norm(st):
    case = st["case"]
    dt, eps, a = _tdt(case["dtype"]), st["eps"], st["res_scale"]
    x, y = st["x"].float(), st["y"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    z, r_post = y, None
    if st["w_post"] is not None:
        r_post = torch.rsqrt((y * y).mean(dim=1, keepdim=True) + eps)
        z = y * r_post * st["w_post"]
    xo = x + a * gate * z
    r_pre = torch.rsqrt((xo * xo).mean(dim=1, keepdim=True) + eps)
    xn = xo * r_pre
    u = xn * st["w_pre"]
    if not case["train"]:
        return xo.to(dt), u.to(dt)
    du = st["du"].float()
    dw_pre = (du * xn).sum(dim=0)
    t = du * st["w_pre"]
    dx = st["dx_out"].float() + r_pre * (t - xn * (t * xn).mean(dim=1, keepdim=True))
    dgz = a * dx
    dz = dgz * gate
    dy, extra = dz, []
    if st["w_post"] is not None:
        yn = y * r_post
        extra.append((dz * yn).sum(dim=0))
        t = dz * st["w_post"]
        dy = r_post * (t - yn * (t * yn).mean(dim=1, keepdim=True))
    if st["gate"] is not None:
        dg = dgz * z
        extra.append(dg.to(dt) if case["gate"] == "token" else dg.sum(dim=0))
    return [xo.to(dt), u.to(dt), dx.to(dt), dy.to(dt), dw_pre] + extra


def _plain_rope(st):
    case = st["case"]
    n, H, d, A = case["n"], case["H"], case["d"], case["axes"]
    half = d // 2
    axis = st["pair_axis"]
    if case["ladder"]:  # each axis runs through its own frequencies
        seen, expo = [0] * A, []
        for a in axis:
            expo.append(seen[a] / axis.count(a))
            seen[a] += 1
    else:
        expo = [j / half for j in range(half)]
    freq = st["theta"] ** (-torch.tensor(expo, dtype=torch.float64, device=DEV))
    pos = st["positions"][torch.tensor(axis, device=DEV)].double().T  # [n, half]
    ang = pos * freq  # far positions: the angle needs 64 bits
    c, s = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if case["mode"] == 2:
        s = -s
    x = st["x"].float()
    if st["bias"] is not None:
        x = x + st["bias"].view(1, H, d)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1).to(_tdt(case["out_dtype"]))


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "norm": _plain_norm, "rope": _plain_rope}[state["case"]["kind"]](state)


# --------------------------------------------------------------- 64-bit values
def exact(case, seed):
    st = _inputs(case, seed)
    if case["kind"] == "attn":
        return _exact_attn(case, st)
    if case["kind"] == "norm":
        return _exact_norm(case, st)
    # rotary: each pair is a complex number times exp(i angle)
    half, A = case["d"] // 2, case["axes"]
    axis = np.asarray(st["pair_axis"])
    expo = np.arange(half) / half
    if case["ladder"]:
        for a in range(A):
            mine = np.flatnonzero(axis == a)
            expo[mine] = np.arange(mine.size) / max(1, mine.size)
    freq = np.power(st["theta"], -expo)
    ang = st["positions"].cpu().numpy()[axis].T.astype(np.float64) * freq[None]
    turn = np.exp(1j * (ang if case["mode"] == 1 else -ang))[:, None, :]
    x = st["x"].double().cpu().numpy()
    if st["bias"] is not None:
        x = x + st["bias"].double().cpu().numpy().reshape(1, case["H"], case["d"])
    z = (x[..., :half] + 1j * x[..., half:]) * turn
    return torch.from_numpy(np.concatenate([z.real, z.imag], axis=-1))


def _exact_attn(case, st):
    # double-precision products take seconds a teraflop on this hardware
    if work(case)["flops"] > 2.5e12:
        return None
    Hq, Hkv, d, P, N, n_q = (case[k] for k in ("Hq", "Hkv", "d", "P", "n_tokens", "n_q"))
    f64 = torch.float64
    b_np, e_np = _spans(case)
    begin, end = torch.from_numpy(b_np).to(DEV)[:, None], torch.from_numpy(e_np).to(DEV)[:, None]
    rows = torch.arange(N - n_q, N, device=DEV)[:, None]
    first = int(b_np.min())
    out_o, out_l, out_dq = [], [], []
    n_pages = st["order"].numel()
    gk = torch.zeros(Hkv, n_pages, P, d, dtype=f64, device=DEV)
    gv = torch.zeros(Hkv, n_pages, P, d, dtype=f64, device=DEV)
    for hq in range(Hq):
        h = hq * Hkv // Hq
        keys = torch.cat([torch.arange(int(p) * P, min(N, (int(p) + 1) * P)) for p in st["sel_cpu"][h]])
        keys = keys[keys >= first].to(DEV)
        q = st["q"][:, hq].to(f64).requires_grad_(case["train"])
        k = st["k"][keys, h].to(f64).requires_grad_(case["train"])
        v = st["v"][keys, h].to(f64).requires_grad_(case["train"])
        with torch.set_grad_enabled(case["train"]):
            s = torch.matmul(q, k.T) * st["scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - st["slopes"][hq].to(f64) * (rows - keys[None]).abs().to(f64)
            s = torch.where((keys[None] >= begin) & (keys[None] < end), s, torch.full_like(s, -math.inf))
            l = torch.logsumexp(s, dim=1)
            o = torch.matmul(torch.exp(s - l[:, None]), v)
        out_o.append(o.detach())
        out_l.append(l.detach())
        if case["train"]:
            dq, dk, dv = torch.autograd.grad(o, (q, k, v), st["do"][:, hq].to(f64))
            out_dq.append(dq)
            gk[h].view(-1, d).index_add_(0, keys, dk)
            gv[h].view(-1, d).index_add_(0, keys, dv)
    res = [torch.stack(out_o, dim=1), torch.stack(out_l)]
    if case["train"]:
        logical = torch.empty(n_pages, dtype=torch.long)
        logical[st["order"]] = torch.arange(n_pages)
        res.append(torch.stack(out_dq, dim=1))
        res += [g[:, logical.to(DEV)].transpose(0, 1).contiguous() for g in (gk, gv)]
    return tuple(res)


def _exact_norm(case, st):
    leaf = {k: st[k].double().requires_grad_(True) for k in ("x", "y", "w_pre", "w_post", "gate")
            if st[k] is not None}

    def rms(t):
        return t / torch.sqrt(t.pow(2).sum(dim=1, keepdim=True) / t.shape[1] + st["eps"])

    branch = leaf["y"]
    if "w_post" in leaf:
        branch = rms(branch) * leaf["w_post"]
    if "gate" in leaf:
        branch = branch * leaf["gate"]
    x_out = leaf["x"] + st["res_scale"] * branch
    u = rms(x_out) * leaf["w_pre"]
    if not case["train"]:
        return x_out.detach(), u.detach()
    names = [k for k in ("x", "y", "w_pre", "w_post", "gate") if k in leaf]
    grads = torch.autograd.grad((x_out, u), [leaf[k] for k in names], (st["dx_out"].double(), st["du"].double()))
    return [x_out.detach(), u.detach()] + list(grads)
