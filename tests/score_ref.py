"""Plain float64 form of the chunk attention with modified scores, and how far a kernel may
be from it: bounds for every output element, from the roundings the kernels make.

One rounding is off by at most half a step of its type relative to the value: 2^-8 in bf16,
2^-24 in fp32.  The tensor-core kernels round P and dA to bf16 before their products
(u_p = 2^-8); the CUDA-core kernels keep them in fp32 (u_p = 2^-24).
"""
from __future__ import annotations

import torch

F64 = torch.float64
U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spans(n_q, q_start, total, key_begin=None, key_end=None):
    pos = torch.arange(q_start, q_start + n_q)
    b = torch.zeros_like(pos) if key_begin is None else key_begin.clamp(min=0)
    e = pos + 1 if key_end is None else key_end.clamp(max=total)
    return pos, b, e


def score_attn(q, k, v, sel, P, q_start, scale, cap=0.0, slopes=None, key_begin=None, key_end=None, do=None,
               total=None, tensor_cores=True):
    """q [n, Hq, d], k and v [total, Hkv, d], sel: per KV head a list of pages.  Returns a dict
    of values (o, lse and with ``do`` dq, dk, dv) and of bounds (o_tol, ...)."""
    n, Hq, d = q.shape
    total = k.shape[0] if total is None else total
    Hkv = k.shape[1]
    G = Hq // Hkv
    u_out = half_step(q.dtype)
    u_p = 2.0 ** -8 if tensor_cores else U32
    pos, b, e = spans(n, q_start, total, key_begin, key_end)
    out = {"o": torch.zeros(n, Hq, d, dtype=F64), "lse": torch.full((Hq, n), -float("inf"), dtype=F64)}
    out["o_tol"], out["lse_tol"] = torch.zeros(n, Hq, d, dtype=F64), torch.zeros(Hq, n, dtype=F64)
    if do is not None:
        for name, shape in (("dq", (n, Hq, d)), ("dk", (total, Hkv, d)), ("dv", (total, Hkv, d))):
            out[name], out[name + "_tol"] = torch.zeros(shape, dtype=F64), torch.zeros(shape, dtype=F64)
    for h in range(Hkv):
        tok = torch.cat([torch.arange(p * P, min(total, (p + 1) * P)) for p in sel[h]] or
                        [torch.zeros(0, dtype=torch.long)])
        kh, vh = k[tok, h].to(F64), v[tok, h].to(F64)
        see = (tok[None] >= b[:, None]) & (tok[None] < e[:, None])
        any_ = see.any(dim=1)
        terms = tok.numel() + 16
        for hq in range(h * G, (h + 1) * G):
            qh = q[:, hq].to(F64)
            a = qh @ kh.T * scale
            t = torch.zeros_like(a)
            s = a
            if cap > 0:
                t = torch.tanh(a / cap)
                s = cap * t
            if slopes is not None:
                s = s - float(slopes[hq]) * (pos[:, None] - tok[None]).abs().to(F64)
            # error of a score: the dot product in fp32, then a few fp32 operations on values
            # no larger than the cap and the bias
            ds = scale * (d + 4) * U32 * (qh.abs() @ kh.abs().T) + 8 * U32 * (s.abs() + a.abs() + cap)
            sm = s.masked_fill(~see, -float("inf"))
            lse = torch.where(any_, torch.logsumexp(sm, dim=1) if tok.numel() else torch.zeros(n, dtype=F64),
                              torch.tensor(-float("inf"), dtype=F64))
            p = torch.where(see, torch.exp(sm - torch.where(any_, lse, torch.zeros_like(lse))[:, None]),
                            torch.zeros_like(sm))
            es = (ds * see).amax(dim=1) if tok.numel() else torch.zeros(n, dtype=F64)
            out["lse"][hq] = lse
            # scores, then a sum of positive terms and its logarithm (2^-20 for the base-2 steps)
            out["lse_tol"][hq] = es + terms * U32 + 2.0 ** -20 + 4 * U32 * lse.abs().nan_to_num(posinf=0.0)
            ep = (2 * es + 2 * terms * U32 + 2.0 ** -20)[:, None]  # relative error of P before rounding
            o = p @ vh
            o_tol = (u_p + ep) * (p @ vh.abs()) + u_out * o.abs()
            out["o"][:, hq], out["o_tol"][:, hq] = o, o_tol
            if do is None:
                continue
            doh = do[:, hq].to(F64)
            dp = doh @ vh.T
            D = (doh * o).sum(dim=1, keepdim=True)
            gate = 1 - t * t
            da = p * (dp - D) * gate
            # D is formed from the rounded O; tanh^2 has an absolute error of a few 2^-24; dP is
            # an fp32 dot product
            dD = (doh.abs() * o_tol).sum(dim=1, keepdim=True) + d * U32 * (doh.abs() * o.abs()).sum(dim=1, keepdim=True)
            ddp = (d + 4) * U32 * (doh.abs() @ vh.abs().T)
            e_da = (u_p + 3 * ep) * da.abs() + p * (dD + ddp) * gate + 16 * U32 * p * (dp - D).abs()
            out["dq"][:, hq] = scale * da @ kh
            out["dq_tol"][:, hq] = scale * ((e_da + terms * U32 * da.abs()) @ kh.abs()) + \
                u_out * (scale * da @ kh).abs() + 8 * U32 * scale * (da.abs() @ kh.abs())
            rows = n * G + 16
            out["dk"].index_put_((tok, torch.tensor(h)), scale * da.T @ qh, accumulate=True)
            out["dv"].index_put_((tok, torch.tensor(h)), p.T @ doh, accumulate=True)
            out["dk_tol"].index_put_((tok, torch.tensor(h)), scale * ((e_da + rows * U32 * da.abs()).T @ qh.abs()),
                                     accumulate=True)
            out["dv_tol"].index_put_((tok, torch.tensor(h)), ((u_p + ep + rows * U32) * p).T @ doh.abs(),
                                     accumulate=True)
    return out


def check(name, got, ref):
    """got (any dtype, any device) against ref[name] within ref[name + '_tol'], element by element."""
    g, r, tol = got.detach().cpu().to(F64), ref[name], ref[name + "_tol"]
    inf = torch.isinf(r)
    assert torch.equal(g[inf], r[inf]), f"{name}: infinities differ"
    assert torch.isfinite(g[~inf]).all(), f"{name}: not finite"
    over = torch.where(inf, torch.zeros_like(r), (g - torch.where(inf, torch.zeros_like(r), r)).abs() - tol)
    over = torch.where(inf, torch.zeros_like(r), over)
    worst = over.max().item() if over.numel() else 0.0
    if worst > 1e-30:
        at = torch.nonzero(over == over.max())[0].tolist()
        raise AssertionError(f"{name}{at}: {g[tuple(at)]:.8g} against {r[tuple(at)]:.8g}, allowed {tol[tuple(at)]:.3g}; "
                             f"{int((over > 1e-30).sum())} of {over.numel()} outside")
