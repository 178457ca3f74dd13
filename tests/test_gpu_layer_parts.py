"""The layer step with its optional parts together - the norms around the previous block with
gate and residual scale, rotary positions in three axes, capped and biased scores, packed
documents with prefixes - against one float64 autograd graph of the same layer."""
import math

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300.layer import LayerStep
from paged_sparse_attention_gb300.pool import PagedKVPool

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def rms(x, w, eps):
    return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w


def turn(x, pos, axis, theta):
    half = x.shape[-1] // 2
    ang = pos[torch.tensor(axis)].to(F64).T * theta ** (-torch.arange(half, dtype=F64) / half)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def layer64(t, cfg, seen):
    """O and the gradients of every leaf; ``seen`` [N, N]: key j is visible to row i."""
    leaf = {k: v.to(F64).requires_grad_(True) for k, v in t.items() if k in
            ("X", "Y", "Wq", "Wk", "Wv", "w_norm", "w_post", "gate", "bq", "bk", "bv")}
    x = leaf["X"]
    if "Y" in leaf:
        x = x + cfg["res_scale"] * leaf["gate"] * rms(leaf["Y"], leaf["w_post"], 1e-6)
    u = rms(x, leaf["w_norm"], 1e-6) if "w_norm" in leaf else x
    N, d, Hq, Hkv = x.shape[0], cfg["d"], cfg["Hq"], cfg["Hkv"]
    q, k, v = ((u @ leaf["W" + c] + leaf["b" + c]).view(N, -1, d) for c in "qkv")
    q, k = (turn(z, t["positions"], cfg["axis"], cfg["theta"]) for z in (q, k))
    k, v = (z.repeat_interleave(Hq // Hkv, dim=1) for z in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
    if cfg["cap"]:
        s = cfg["cap"] * torch.tanh(s / cfg["cap"])
    i = torch.arange(N)
    s = s - t["slopes"].to(F64)[:, None, None] * (i[:, None] - i[None]).abs()
    p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
    o = torch.einsum("hij,jhd->ihd", p, v)
    names = list(leaf)
    outs, grads = [o], [t["dO"].to(F64)]
    if "w_norm" in leaf:
        outs.append(x)
        grads.append(t["dX_out"].to(F64))
    g = torch.autograd.grad(outs, [leaf[n] for n in names], grads)
    return o.detach(), x.detach(), dict(zip(names, g))


@pytest.mark.parametrize("name,cfg", [
    ("bf16", dict(dtype=torch.bfloat16, N=700, chunk=256, P=128, Hq=4, Hkv=2, d=128, Dm=256, block=True)),
    ("bf16_small_pages", dict(dtype=torch.bfloat16, N=300, chunk=128, P=32, Hq=4, Hkv=1, d=64, Dm=128, block=False)),
    ("fp32", dict(dtype=torch.float32, N=330, chunk=128, P=64, Hq=2, Hkv=1, d=64, Dm=96, block=True)),
])
def test_layer_with_all_parts(name, cfg):
    cfg = dict(cfg, cap=8.0, theta=1e4, res_scale=0.8, axis=[j % 3 for j in range(cfg["d"] // 2)])
    dt, N, chunk, P, Hq, Hkv, d, Dm = (cfg[k] for k in ("dtype", "N", "chunk", "P", "Hq", "Hkv", "d", "Dm"))
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"X": rn(N, Dm).to(dt), "dO": rn(N, Hq, d).to(dt), "dX_out": (0.1 * rn(N, Dm)).to(dt),
         "w_norm": 1 + 0.2 * rn(Dm), "slopes": 2.0 ** -(1.0 + torch.arange(Hq)),
         "positions": torch.stack([1000 + torch.arange(N) // 16, torch.arange(N) // 4 % 4, torch.arange(N) % 4])}
    for c, H in (("q", Hq), ("k", Hkv), ("v", Hkv)):
        t["W" + c] = (rn(Dm, H * d) / math.sqrt(Dm)).to(dt)
        t["b" + c] = 0.1 * rn(H * d)
    if cfg["block"]:
        t.update(Y=rn(N, Dm).to(dt), w_post=1 + 0.2 * rn(Dm), gate=0.5 + 0.2 * rn(Dm))
    cuts = [0, 90, 91, 260, N - 5, N]
    prefix = [30, 1, 100, 60, 0]
    # what the rows see: their document up to themselves, its prefix, chunks up to their own
    seen = torch.zeros(N, N, dtype=torch.bool)
    for c in range(len(cuts) - 1):
        for i in range(cuts[c], cuts[c + 1]):
            end = max(i + 1, min(cuts[c] + prefix[c], cuts[c + 1]))
            seen[i, cuts[c]:min(end, (i // chunk + 1) * chunk)] = True
    o64, x64, g64 = layer64(t, cfg, seen)
    dev = torch.device("cuda")
    up = {k: v.to(dev) for k, v in t.items()}
    n_pages = -(-N // P)
    pool = PagedKVPool(Hq, Hkv, d, P, n_pages, n_pages, dt, dev,
                       page_order=torch.randperm(n_pages, generator=g).to(torch.int32))
    step = LayerStep(pool, up["Wq"], up["Wk"], up["Wv"], up["bq"], up["bk"], up["bv"], chunk=chunk,
                     theta=cfg["theta"], softcap=cfg["cap"], slopes=up["slopes"], pair_axis=cfg["axis"],
                     w_norm=up["w_norm"], w_post=up.get("w_post"), gate=up.get("gate"), res_scale=cfg["res_scale"])
    out = step.run(up["X"], up["dO"], Y=up.get("Y"), dX_out=up["dX_out"], positions=up["positions"],
                   doc_start=torch.tensor(cuts, device=dev), prefix_len=torch.tensor(prefix, device=dev))
    assert L.oomb_check(pool.handle) == 0
    # about nine roundings to bf16 lie between the leaves and a gradient (normed input, q/k/v,
    # P, O, dA, dq, du, dx); each is at most 2^-8 and 2^-8 / sqrt(3) in the mean: 0.7 % together
    tol = 1e-5 if dt == torch.float32 else 1e-2

    def rel(a, b):
        return ((a.to(F64).cpu() - b).norm() / b.norm()).item()

    assert rel(torch.cat(out["O"]), o64) < tol
    assert rel(out["X_out"], x64) < tol
    for key, ref in (("dX", "X"), ("dY", "Y"), ("dWq", "Wq"), ("dWk", "Wk"), ("dWv", "Wv"), ("dbq", "bq"),
                     ("dbv", "bv"), ("dw_norm", "w_norm"), ("dw_post", "w_post"), ("dgate", "gate")):
        if ref in g64:
            assert out[key].shape == t[ref].shape and rel(out[key], g64[ref]) < tol, (key, rel(out[key], g64[ref]))
    pool.close()


def test_parts_that_need_one_another():
    dev = torch.device("cuda")
    pool = PagedKVPool(2, 1, 64, 64, 2, 2, torch.float32, dev)
    W = torch.zeros(8, 128, device=dev), torch.zeros(8, 64, device=dev), torch.zeros(8, 64, device=dev)
    one = torch.ones(8, device=dev)
    X, dO = torch.zeros(64, 8, device=dev), torch.zeros(64, 2, 64, device=dev)
    with pytest.raises(ValueError):
        LayerStep(pool, *W, gate=one)
    with pytest.raises(ValueError):
        LayerStep(pool, *W, chunk=64, pair_axis=[0] * 32).run(X, dO)
    with pytest.raises(ValueError):
        LayerStep(pool, *W, chunk=64).run(X, dO, Y=X)
    with pytest.raises(ValueError):
        LayerStep(pool, *W, chunk=64, w_norm=one, w_post=one).run(X, dO)
    with pytest.raises(ValueError):
        LayerStep(pool, *W, chunk=64).run(X, dO, prefix_len=torch.zeros(1, dtype=torch.int64, device=dev))
    pool.close()
