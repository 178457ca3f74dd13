"""Embeddings, an attention layer, the last norm and the loss run together, against float64 autograd."""
import math

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300.ends import ModelEnds
from paged_sparse_attention_gb300.layer import LayerStep
from paged_sparse_attention_gb300.pool import PagedKVPool

pytestmark = pytest.mark.gpu

BF, FP, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def rotate(t, theta=1e6):
    """Rotate-half rotary embedding of [N, H, d] at positions 0.."""
    N, _, d = t.shape
    ang = torch.arange(N, dtype=F64)[:, None] * theta ** (-torch.arange(0, d, 2, dtype=F64) / d)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = t[..., :d // 2], t[..., d // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def model(p, tokens, targets, weights, scale, softcap, Hq, Hkv, d):
    """scale * sum of the weighted losses, and the losses: the same model in float64."""
    N = tokens.numel()
    X = torch.where((tokens >= 0)[:, None], p["table"][tokens.clamp_min(0)] * 1.5, torch.zeros((), dtype=F64))
    q, k, v = (rotate((X @ p[w]).view(N, H, d)) if w != "Wv" else (X @ p[w]).view(N, H, d)
               for w, H in (("Wq", Hq), ("Wk", Hkv), ("Wv", Hkv)))
    k, v = k.repeat_interleave(Hq // Hkv, 1), v.repeat_interleave(Hq // Hkv, 1)
    att = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
    att = att.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf")).softmax(-1)
    h = torch.einsum("hij,jhd->ihd", att, v).reshape(N, Hq * d)
    if "w" in p:
        c = h - h.mean(1, keepdim=True)
        h = c * torch.rsqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["w"] + p["b"]
    z = h @ p.get("head", p["table"]).t()
    if softcap:
        z = softcap * torch.tanh(z / softcap)
    loss = torch.where(targets >= 0, torch.logsumexp(z, 1) - z[torch.arange(N), targets.clamp_min(0)],
                       torch.zeros((), dtype=F64))
    return scale * (loss * weights).sum(), loss


@pytest.mark.parametrize("tied,norm,softcap", [(True, True, 0.0), (False, True, 20.0), (False, False, 0.0)])
@pytest.mark.parametrize("dtype,tol", [(FP, 2e-5), (BF, 2e-2)])
def test_a_model_chunk_by_chunk(dtype, tol, tied, norm, softcap):
    Hq, Hkv, d, P, N, chunk, V = 2, 1, 64, 64, 300, 128, 517
    Dm = Hq * d
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"table": rn(V, Dm).mul(0.7).to(dtype)}
    for w, H in (("Wq", Hq), ("Wk", Hkv), ("Wv", Hkv)):
        p[w] = (rn(Dm, H * d) / math.sqrt(Dm)).to(dtype)
    if norm:
        p["w"], p["b"] = 1 + 0.2 * rn(Dm), 0.2 * rn(Dm)
    if not tied:
        p["head"] = (rn(V, Dm) / math.sqrt(Dm)).to(dtype)
    tokens = (float(V) ** torch.rand(N, generator=g, dtype=F64)).floor().long() - 1
    targets = torch.cat([tokens[1:], torch.tensor([-1])])
    targets[40:200] = -1  # a prompt, over a chunk's end
    tokens[250:260] = -1
    weights = 0.5 + torch.rand(N, generator=g)
    scale = 1.0 / 139
    f = {k: v.to(F64).requires_grad_() for k, v in p.items()}
    total, want_loss = model(f, tokens, targets, weights.to(F64), scale, softcap, Hq, Hkv, d)
    total.backward()

    c = {k: v.cuda() for k, v in p.items()}
    n_pages = -(-N // P)
    pool = PagedKVPool(Hq, Hkv, d, P, n_pages, n_pages, dtype, torch.device("cuda", torch.cuda.current_device()))
    layer = LayerStep(pool, c["Wq"], c["Wk"], c["Wv"], chunk=chunk)
    ends = ModelEnds(c["table"], head=c.get("head"), w_norm=c.get("w"), b_norm=c.get("b"), chunk=chunk, scale=1.5,
                     softcap=softcap)
    tok, tgt, wts = tokens.cuda(), targets.cuda(), weights.cuda()
    loss = torch.full((N,), float("nan"), device="cuda")
    for _ in range(2):  # a second step from zeroed gradients gives the same
        ends.zero_grad()
        X = ends.embed(tok)
        out = layer.run(X, ends.behind(tgt, loss, wts, scale))
        ends.embed_grad(tok, out["dX"])
        ends.check()
        L.oomb_check(pool.handle)
        got = {"table": ends.d_table, "Wq": out["dWq"], "Wk": out["dWk"], "Wv": out["dWv"]}
        if norm:
            got.update(w=ends.dw_norm, b=ends.db_norm)
        if not tied:
            got["head"] = ends.d_head
        # relative errors over whole tensors: fp32 sums of at most 517 terms a product through six of them;
        # bf16 tensors rounded to 2^-8 at each of about ten stages, whose errors add as squares or nearly so
        assert (loss.cpu().to(F64) - want_loss.detach()).norm() <= tol * want_loss.detach().norm()
        for k, v in got.items():
            e = (v.cpu().to(F64) - f[k].grad).norm() / f[k].grad.norm()
            assert e <= tol, (k, float(e))


def test_evaluation_without_gradients_and_refusals():
    g = torch.Generator().manual_seed(1)
    table = torch.randn(100, 64, generator=g).cuda()
    ends = ModelEnds(table, w_norm=torch.ones(64, device="cuda"), chunk=50)
    h, t = torch.randn(50, 64, generator=g).cuda(), torch.randint(0, 100, (50,), generator=g).cuda()
    a, b = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    assert ends.chunk_loss(h, t, a, grads=False) is None
    assert (ends.d_table == 0).all() and (ends.dw_norm == 0).all()
    assert ends.chunk_loss(h, t, b) is not None and torch.equal(a, b)
    with pytest.raises(ValueError, match="at most 50"):
        ends.chunk_loss(torch.zeros(51, 64, device="cuda"), t, a)
    ends.embed(torch.tensor([3, 100], device="cuda"))
    with pytest.raises(L.OombError, match="0x20"):
        ends.check()
    ends.check()
