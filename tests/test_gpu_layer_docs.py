"""The layer step on packed documents with less than every page: a local window, and pages that
the caller gives - against one float64 autograd graph; the key bias' gradient among them."""
import math

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300.layer import LayerStep
from paged_sparse_attention_gb300.pool import PagedKVPool
from test_gpu_layer_parts import turn

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def layer64(t, cfg, seen):
    """O, the gradients of the leaves, and of the key projections before they are summed."""
    leaf = {n: t[n].to(F64).requires_grad_(True) for n in ("X", "Wq", "Wk", "Wv", "bq", "bk", "bv")}
    N, d, G = t["X"].shape[0], cfg["d"], cfg["Hq"] // cfg["Hkv"]
    q, k, v = ((leaf["X"] @ leaf["W" + c] + leaf["b" + c]).view(N, -1, d) for c in "qkv")
    pos = torch.arange(N)[None]
    qr, kr = (turn(z, pos, [0] * (d // 2), cfg["theta"]) for z in (q, k))
    kr, vr = (z.repeat_interleave(G, dim=1) for z in (kr, v))
    s = torch.einsum("ihd,jhd->hij", qr, kr) / math.sqrt(d)
    s = cfg["cap"] * torch.tanh(s / cfg["cap"])
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~seen, -math.inf), -1), vr)
    g = torch.autograd.grad(o, [*leaf.values(), k], t["dO"].to(F64))
    return o.detach(), dict(zip(leaf, g)), g[-1]


@pytest.mark.parametrize("kind", ["window", "given"])
@pytest.mark.parametrize("cfg", [
    dict(dtype=torch.bfloat16, N=1000, chunk=256, P=128, Hq=4, Hkv=2, d=128, Dm=256),
    dict(dtype=torch.float32, N=330, chunk=128, P=32, Hq=2, Hkv=1, d=64, Dm=96)], ids=["bf16", "fp32"])
def test_documents_and_pages(cfg, kind):
    cfg = dict(cfg, cap=8.0, theta=1e4)
    dt, N, chunk, P, Hq, Hkv, d, Dm = (cfg[k] for k in ("dtype", "N", "chunk", "P", "Hq", "Hkv", "d", "Dm"))
    g = torch.Generator().manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"X": rn(N, Dm).to(dt), "dO": rn(N, Hq, d).to(dt)}
    for c, H in (("q", Hq), ("k", Hkv), ("v", Hkv)):
        t["W" + c] = (rn(Dm, H * d) / math.sqrt(Dm)).to(dt)
        t["b" + c] = 0.3 * rn(H * d)
    cuts = [0, N // 10, N // 2 + 3, N]
    window = 1
    doc = torch.searchsorted(torch.tensor(cuts), torch.arange(N), right=True) - 1
    start = torch.tensor(cuts)[doc]
    pages = []  # of each chunk
    for s in range(0, N, chunk):
        own0, end = s // P, -(-min(s + chunk, N) // P)
        first = max(0, own0 - window) if kind == "window" else int(start[s]) // P  # given: every other document page
        pages.append([p for p in range(first, end) if kind == "window" or p >= own0 or (p - first) % 2 == 0])
    seen = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        for p in pages[i // chunk]:
            seen[i, max(p * P, int(start[i])):min((p + 1) * P, i + 1)] = True
    o64, g64, gk = layer64(t, cfg, seen)
    dev = torch.device("cuda")
    up = {k: v.to(dev) for k, v in t.items()}
    n_pages = -(-N // P)
    pool = PagedKVPool(Hq, Hkv, d, P, n_pages, n_pages, dt, dev)
    kw = dict(window=window, n_sink=0) if kind == "window" else dict(top_k=1)
    step = LayerStep(pool, up["Wq"], up["Wk"], up["Wv"], up["bq"], up["bk"], up["bv"], chunk=chunk, theta=cfg["theta"],
                     softcap=cfg["cap"], **kw)
    given = None
    if kind == "given":
        given = [(torch.tensor([p] * Hkv, dtype=torch.int32, device=dev),
                  torch.full((Hkv,), len(p), dtype=torch.int32, device=dev)) for p in pages]
    out = step.run(up["X"], up["dO"], sel_override=given, doc_start=torch.tensor(cuts, device=dev))
    assert L.oomb_check(pool.handle) == 0
    # six roundings to bf16 between the leaves and a gradient (q/k/v, P, O, dA, dq, the weights' own
    # cast), each at most 2^-8 and 2^-8 / sqrt(3) in the mean: 0.6 % together
    tol = 1e-5 if dt == torch.float32 else 1e-2

    def rel(a, b):
        return ((a.to(F64).cpu() - b).norm() / b.norm()).item()

    assert rel(torch.cat(out["O"]), o64) < tol
    for name in ("X", "Wq", "Wk", "Wv", "bq", "bv"):
        assert rel(out["d" + name], g64[name]) < tol, (name, rel(out["d" + name], g64[name]))
    # the key bias' gradient is a sum of terms that nearly cancel: held to the size of the terms
    err = (out["dbk"].to(F64).cpu() - g64["bk"]).abs()
    assert (err <= tol * gk.abs().sum(0).view(-1)).all() and g64["bk"].abs().max() > 0
    pool.close()


def test_prefixes_that_cross_a_chunk_are_told():
    dev = torch.device("cuda")
    pool = PagedKVPool(2, 1, 64, 32, 4, 4, torch.float32, dev)
    W = torch.zeros(8, 128, device=dev), torch.zeros(8, 64, device=dev), torch.zeros(8, 64, device=dev)
    X, dO = torch.zeros(100, 8, device=dev), torch.zeros(100, 2, 64, device=dev)
    docs, pre = torch.tensor([0, 20, 60, 70, 100], device=dev), torch.tensor([20, 13, 200, 26], device=dev)
    step = LayerStep(pool, *W, chunk=32)
    assert step.run(X, dO, doc_start=docs, prefix_len=pre)["prefix_cut"].tolist() == [False, True, True, False]
    assert "prefix_cut" not in step.run(X, dO, doc_start=docs)
    assert L.oomb_check(pool.handle) == 0
    pool.close()
