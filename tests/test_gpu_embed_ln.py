"""Token embeddings with their gradient by sorted tokens, and layer norm, on the GPU against float64."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from ends_ref import U32, check, half_step

pytestmark = pytest.mark.gpu

BF, FP, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ embeddings
def embed(tokens, table, d_out, scale, accumulate, base, ws=None):
    n, (V, D) = tokens.numel(), table.shape
    t, tab, d = tokens.cuda(), table.cuda(), d_out.cuda()
    out = torch.full((n, D), float("nan"), dtype=table.dtype, device="cuda")
    grad = base.cuda().clone()
    err = word()
    if ws is None:
        ws = torch.full((L.oomb_embed_workspace(n, D),), 255, dtype=torch.uint8, device="cuda")
    L.oomb_embed_fwd(t, tab, out, err, scale=scale)
    L.oomb_embed_bwd(t, d, grad, ws, err, scale=scale, accumulate=accumulate)
    assert L.oomb_word_check(err) == 0
    return out.cpu(), grad.cpu()


def check_embed(tokens, table, d_out, scale=1.0, accumulate=True, base=None, **kw):
    V, D = table.shape
    if base is None:
        base = torch.randn(V, D, generator=torch.Generator().manual_seed(3))
    out, grad = embed(tokens, table, d_out, scale, accumulate, base, **kw)
    real = tokens >= 0
    at = tokens.clamp_min(0)
    want = torch.where(real[:, None], scale * table.to(F64)[at], torch.zeros((), dtype=F64))
    assert ((out.to(F64) - want).abs() <= (half_step(table.dtype) + U32) * want.abs()).all()
    assert (out[~real] == 0).all()
    rows = d_out.to(F64)[real]
    total = torch.zeros(V, D, dtype=F64).index_add_(0, at[real], rows)
    mag = torch.zeros(V, D, dtype=F64).index_add_(0, at[real], rows.abs())
    count = torch.bincount(at[real], minlength=V)
    named = count > 0
    # a sum of m fp32 terms in pieces: fewer than m + 8 roundings, then the scale and the addition
    tol = (count[:, None] + 16) * U32 * abs(scale) * mag + 2 * U32 * base.abs().to(F64)
    ref = (base.to(F64) if accumulate else 0.0) + scale * total
    assert ((grad.to(F64) - ref).abs()[named] <= tol[named]).all()
    assert torch.equal(grad[~named], base[~named])
    return grad


def ids(kind, n, V, g):
    if kind == "same":
        return torch.full((n,), V // 2)
    if kind == "few":
        return torch.randint(0, min(V, 3), (n,), generator=g)
    if kind == "distinct":
        return torch.randperm(max(n, V), generator=g)[:n] % V
    if kind == "none":
        return torch.full((n,), -1)
    u = torch.rand(n, generator=g, dtype=F64)
    t = (float(V) ** u).floor().long() - 1
    if kind == "padded":
        t[torch.rand(n, generator=g) < 0.3] = -1
        t[n // 2] = -(2 ** 62)
    return t


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", ["same", "few", "distinct", "spread", "padded", "none"])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (2, 50, 7), (63, 50, 8), (64, 20, 33), (65, 20, 64), (129, 1000, 40),
                                   (1000, 300, 1000), (4096, 5000, 24), (8192, 700, 16), (8193, 700, 9),
                                   (20000, 3000, 12)])
def test_embed_matches(dtype, kind, n, V, D):
    g = torch.Generator().manual_seed(n + V)
    t = ids(kind, n, V, g)
    check_embed(t, torch.randn(V, D, generator=g).to(dtype), torch.randn(n, D, generator=g).to(dtype),
                scale=1.0 if n % 2 else 45.25)


@pytest.mark.parametrize("kind", ["same", "few", "distinct", "spread", "padded", "none"])
@pytest.mark.parametrize("n", [1023, 4095, 4097, 5120, 5121, 28672, 28673, 70001])
def test_embed_orders(n, kind):
    """On both sides of the ways to the tokens' order; small vocabularies and ones of few bits to spare."""
    g = torch.Generator().manual_seed(n)
    for V, D in ((511, 8), (70000, 3)):
        check_embed(ids(kind, n, V, g), torch.randn(V, D, generator=g).to(BF), torch.randn(n, D, generator=g).to(BF))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 34])
def test_embed_few_rows(dtype, n):
    """On both sides of the gradient in one launch."""
    g = torch.Generator().manual_seed(n)
    for kind, V, D in (("few", 9, 264), ("distinct", 50, 33), ("padded", 2 ** 20, 8), ("same", 3, 5000), ("none", 5, 8)):
        t = ids(kind, n, V, g)
        for acc in (True, False):
            check_embed(t, torch.randn(V, D, generator=g).to(dtype), torch.randn(n, D, generator=g).to(dtype), scale=0.3,
                        accumulate=acc)


@pytest.mark.parametrize("runs", [[16], [17], [33], [15, 2, 15], [5, 600, 5], [513, 513], [64], [65], [128], [129], [1, 64, 1], [63, 65, 64], [16, 16, 16, 200], [3, 300, 2, 70, 64],
                                  [65, 65, 65, 65], [1] * 40 + [90] + [1] * 20 + [66]])
def test_runs_around_the_piece(runs):
    """Tokens that occur a window's rows, one more, two windows; long runs next to one another."""
    g = torch.Generator().manual_seed(len(runs))
    t = torch.cat([torch.full((m,), 2 * i) for i, m in enumerate(runs)])
    n, V = t.numel(), 2 * len(runs) + 3
    for order in (torch.arange(n), torch.randperm(n, generator=g)):
        check_embed(t[order], torch.randn(V, 72, generator=g).to(BF), torch.randn(n, 72, generator=g).to(BF))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_wide_rows_written_not_added(dtype):
    g = torch.Generator().manual_seed(1)
    for D in (3584, 5000, 16387):
        t = ids("padded", 300, 90, g)
        check_embed(t, torch.randn(90, D, generator=g).to(dtype), torch.randn(300, D, generator=g).to(dtype),
                    scale=0.5, accumulate=False)


def test_rows_without_a_token_are_not_read():
    g = torch.Generator().manual_seed(2)
    t = ids("padded", 500, 60, g)
    d = torch.randn(500, 32, generator=g)
    d[t < 0] = float("nan")
    base = torch.zeros(60, 32)
    _, grad = embed(t, torch.randn(60, 32, generator=g), d, 1.0, True, base)
    assert torch.isfinite(grad).all()


def test_the_same_bits_on_every_run_and_the_order_of_rows():
    g = torch.Generator().manual_seed(4)
    t, d = ids("spread", 9000, 500, g), torch.randn(9000, 40, generator=g)
    tab, base = torch.randn(500, 40, generator=g), torch.zeros(500, 40)
    a = embed(t, tab, d, 1.0, True, base)[1]
    assert torch.equal(a, embed(t, tab, d, 1.0, True, base)[1])
    # a token's rows within 16 sorted ones are added one after another
    t = torch.arange(32) % 2
    one = torch.zeros(40)
    for i in range(0, 32, 2):
        one += d[i]
    assert torch.equal(embed(t, tab, d[:32], 1.0, True, base)[1][0], one)


def test_a_token_behind_the_vocabulary_is_told():
    g = torch.Generator().manual_seed(5)
    t = torch.randint(0, 30, (70,), generator=g)
    bad = t.clone()
    bad[3], bad[69] = 30, 2 ** 33 + 1
    ok = torch.where(bad >= 30, torch.full_like(bad, -1), bad)
    tab, d, base = torch.randn(30, 24, generator=g), torch.randn(70, 24, generator=g), torch.zeros(30, 24)
    want = embed(ok, tab, d, 1.0, True, base)
    err = word()
    out, grad = torch.empty(70, 24, device="cuda"), base.cuda()
    ws = torch.empty(L.oomb_embed_workspace(70, 24), dtype=torch.uint8, device="cuda")
    for call in (lambda: L.oomb_embed_fwd(bad.cuda(), tab.cuda(), out, err),
                 lambda: L.oomb_embed_bwd(bad.cuda(), d.cuda(), grad, ws, err, accumulate=True)):
        call()
        with pytest.raises(L.OombError, match="0x20"):
            L.oomb_word_check(err)
    assert torch.equal(out.cpu(), want[0]) and torch.equal(grad.cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_embed_off_16_bytes_and_workspace(dtype):
    g = torch.Generator().manual_seed(6)
    V, D, n = 40, 64, 300
    t = ids("few", n, V, g)
    tab, d, base = torch.randn(V, D, generator=g).to(dtype), torch.randn(n, D, generator=g).to(dtype), torch.zeros(V, D)
    want = embed(t, tab, d, 1.0, True, base)
    off = lambda s, dt: torch.empty(s.numel() + 1, dtype=dt, device="cuda")[1:].view(s.shape)  # noqa: E731
    out, grad, err = off(d, dtype), off(base, FP).zero_(), word()
    size = L.oomb_embed_workspace(n, D)
    ws = torch.full((size + 512,), 171, dtype=torch.uint8, device="cuda")
    L.oomb_embed_fwd(t.cuda(), off(tab, dtype).copy_(tab), out, err)
    L.oomb_embed_bwd(t.cuda(), off(d, dtype).copy_(d), grad, ws[:size], err, accumulate=True)
    assert torch.equal(out.cpu(), want[0]) and torch.equal(grad.cpu(), want[1])
    assert (ws[size:] == 171).all()
    sizes = [L.oomb_embed_workspace(m, D) for m in (1, 64, 65, 100, 8192, 8193, 70000)]
    assert sizes == sorted(sizes)


def test_embed_graph_replays_with_new_tokens():
    g = torch.Generator().manual_seed(7)
    V, D, n = 400, 128, 9000
    t, d = ids("padded", n, V, g).cuda(), torch.randn(n, D, generator=g).to(BF).cuda()
    tab, grad = torch.randn(V, D, generator=g).to(BF).cuda(), torch.zeros(V, D, device="cuda")
    out, err = torch.empty(n, D, dtype=BF, device="cuda"), word()
    ws = torch.empty(L.oomb_embed_workspace(n, D), dtype=torch.uint8, device="cuda")

    def step():
        L.oomb_embed_fwd(t, tab, out, err)
        L.oomb_embed_bwd(t, d, grad, ws, err, accumulate=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    grad.zero_()
    new = ids("spread", n, V, g)
    t.copy_(new)
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    base = torch.zeros(V, D)
    once = embed(new, tab.cpu(), d.cpu(), 1.0, True, base)
    twice = embed(new, tab.cpu(), d.cpu(), 1.0, True, once[1])
    assert torch.equal(out.cpu(), once[0]) and torch.equal(grad.cpu(), twice[1])


def test_embed_offsets_past_32_bits():
    V, D = 1_100_003, 2048
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    tab = torch.zeros(V, D, dtype=BF, device="cuda")
    tab[-1], tab[V // 2] = 3.0, 5.0
    t = torch.tensor([V - 1, 0, V // 2, V - 1], device="cuda")
    out, err = torch.empty(4, D, dtype=BF, device="cuda"), word()
    L.oomb_embed_fwd(t, tab, out, err)
    assert (out == torch.tensor([3.0, 0.0, 5.0, 3.0], device="cuda")[:, None]).all()
    del tab
    grad = torch.zeros(V, D, device="cuda")
    ws = torch.empty(L.oomb_embed_workspace(4, D), dtype=torch.uint8, device="cuda")
    d = torch.ones(4, D, dtype=BF, device="cuda")
    L.oomb_embed_bwd(t, d, grad, ws, err, accumulate=True)
    assert (grad[-1] == 2).all() and (grad[0] == 1).all() and (grad[V // 2] == 1).all()
    assert float(grad.sum(dtype=torch.float64)) == 4 * D
    assert L.oomb_word_check(err) == 0


# ------------------------------------------------------------------ layer norm
# fp32 roundings on the way to an element: at most 32 terms a thread, 12 steps of the block's sum,
# and a dozen products
OPS = 64 * U32


def ln_make(n, D, dtype, weight=True, bias=True, through=True, shift=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = {"x": (torch.randn(n, D, generator=g) * 3 + shift).to(dtype), "dy": torch.randn(n, D, generator=g).to(dtype)}
    t["w"] = 1 + 0.3 * torch.randn(D, generator=g) if weight else None
    t["b"] = 0.3 * torch.randn(D, generator=g) if bias else None
    t["dx_out"] = torch.randn(n, D, generator=g).to(dtype) if through else None
    return t


def ln_reference(t, eps, dtype):
    f = {k: None if v is None else v.to(F64) for k, v in t.items()}
    x, n, D = f["x"], *t["x"].shape
    half = half_step(dtype)
    w = torch.ones(D, dtype=F64) if f["w"] is None else f["w"]
    b = torch.zeros(D, dtype=F64) if f["b"] is None else f["b"]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + eps)
    xn = c * r
    e_mean = OPS * x.abs().mean(1, keepdim=True)
    # of xn: the mean's error and a rounding of the difference, then the variance's (which a wrong mean
    # raises by its square only) and the products'
    e_xn = (e_mean + U32 * (x.abs() + mean.abs())) * r * 1.01 + (e_mean * r) ** 2 * xn.abs() + 2 * OPS * xn.abs()
    ref = {"out": xn * w + b}
    tol = {"out": half * ref["out"].abs() + e_xn * w.abs() + 2 * U32 * (xn * w).abs() + U32 * b.abs()}
    dy = f["dy"]
    q = dy * w
    m0, m1 = q.mean(1, keepdim=True), (q * xn).mean(1, keepdim=True)
    v = r * (q - m0 - xn * m1)
    e_m0 = OPS * q.abs().mean(1, keepdim=True)
    e_m1 = (q.abs() * e_xn).mean(1, keepdim=True) + OPS * (q * xn).abs().mean(1, keepdim=True)
    e_r = 2 * OPS + (e_mean * r) ** 2
    dx = v if f["dx_out"] is None else v + f["dx_out"]
    ref["dx"] = dx
    tol["dx"] = (half + 2 * U32) * dx.abs() + e_r * v.abs() + r * (
        e_m0 + xn.abs() * e_m1 + e_xn * m1.abs() + 4 * U32 * (q.abs() + m0.abs() + (xn * m1).abs()))
    ref["dw"], ref["db"] = (dy * xn).sum(0), dy.sum(0)
    tol["dw"] = (dy.abs() * e_xn).sum(0) + (n + 32) * U32 * (dy * xn).abs().sum(0)
    tol["db"] = (n + 32) * U32 * dy.abs().sum(0)
    return ref, tol


def ln_run(t, eps, accumulate=False, base=None):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    n, D = t["x"].shape
    new = lambda: torch.full((n, D), float("nan"), dtype=t["x"].dtype, device="cuda")  # noqa: E731
    vec = lambda: torch.full((D,), float("nan") if base is None else base, device="cuda")  # noqa: E731
    out = {"out": new(), "dx": new(), "dw": vec(), "db": vec()}
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    L.oomb_layer_norm_fwd(d["x"], d["w"], d["b"], out["out"], eps=eps, mean=mean, rstd=rstd)
    ws = torch.empty(L.oomb_layer_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], out["dx"], dw=out["dw"], db=out["db"],
                          dx_out=d["dx_out"], accumulate=accumulate, workspace=ws)
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 31, 64, 256, 1000, 1023, 1537, 3584, 4104, 8192, 8200, 9001, 16384])
@pytest.mark.parametrize("parts", [(True, True, True), (False, False, False), (True, False, True)])
def test_layer_norm_matches(dtype, D, parts):
    t = ln_make(37 if D < 4000 else 5, D, dtype, *parts, seed=D)
    ref, tol = ln_reference(t, 1e-5, dtype)
    check(ln_run(t, 1e-5), ref, tol)


@pytest.mark.parametrize("dtype,n,D", [(BF, 1, 3584), (BF, 1300, 3584), (FP, 3000, 257), (BF, 5000, 64), (FP, 700, 5121),
                                       (BF, 900, 12000)])
def test_layer_norm_many_rows(dtype, n, D):
    t = ln_make(n, D, dtype, seed=n)
    ref, tol = ln_reference(t, 1e-5, dtype)
    check(ln_run(t, 1e-5), ref, tol)


def test_a_mean_far_above_the_spread():
    """Rows at 1000 with a spread of one: squares of the values would lose the variance."""
    t = ln_make(9, 1024, FP, seed=3)
    t["x"] = t["x"] / 3 + 1000
    ref, tol = ln_reference(t, 1e-5, FP)
    check(ln_run(t, 1e-5), ref, tol)


def test_constant_rows_and_no_eps():
    t = ln_make(4, 128, FP, seed=4)
    t["x"][:] = 0.5
    ref, tol = ln_reference(t, 1e-5, FP)
    check(ln_run(t, 1e-5), ref, tol)
    t = ln_make(4, 128, BF, seed=4)
    ref, tol = ln_reference(t, 0.0, BF)
    check(ln_run(t, 0.0), ref, tol)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33])
def test_layer_norm_few_rows_accumulate(n):
    """Up to 16 rows are one block's, which adds to the parameter gradients itself; one gradient alone."""
    for D in (40, 2056, 5000):
        t = ln_make(n, D, BF, seed=n)
        ref, tol = ln_reference(t, 1e-5, BF)
        a, c = ln_run(t, 1e-5), ln_run(t, 1e-5, accumulate=True, base=2.0)
        check(a, ref, tol)
        for k in ("dw", "db"):
            assert torch.equal(c[k], a[k] + 2.0)
        d = {k: v.cuda() for k, v in t.items()}
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        L.oomb_layer_norm_fwd(d["x"], d["w"], d["b"], torch.empty_like(d["x"]), mean=mean, rstd=rstd)
        ws = torch.empty(L.oomb_layer_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
        for key in ("dw", "db", None):
            g = torch.full((D,), 7.0, device="cuda")
            L.oomb_layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], torch.empty_like(d["x"]), dx_out=d["dx_out"],
                                  workspace=ws, **({key: g} if key else {}))
            assert torch.equal(g, a[key] if key else torch.full_like(g, 7.0))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [3584, 1001, 9000])
def test_layer_norm_accumulates_repeats_and_works_in_place(dtype, D):
    t = ln_make(400, D, dtype, seed=5)
    a, b = ln_run(t, 1e-5), ln_run(t, 1e-5)
    c = ln_run(t, 1e-5, accumulate=True, base=2.0)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    for k in ("dw", "db"):
        assert torch.equal(c[k], a[k] + 2.0)
    d = {k: v.cuda() for k, v in t.items()}
    x = d["x"].clone()
    mean, rstd = torch.empty(400, device="cuda"), torch.empty(400, device="cuda")
    L.oomb_layer_norm_fwd(x, d["w"], d["b"], x, eps=1e-5, mean=mean, rstd=rstd)
    assert torch.equal(x, a["out"])
    ws = torch.empty(L.oomb_layer_norm_workspace(400, D), dtype=torch.uint8, device="cuda")
    g = d["dx_out"].clone()
    L.oomb_layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], g, dx_out=g, workspace=ws)
    assert torch.equal(g, a["dx"])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_layer_norm_off_16_bytes(dtype):
    n, D = 50, 256
    t = ln_make(n, D, dtype, seed=6)
    off = lambda s: torch.empty(s.numel() + 1, dtype=s.dtype, device="cuda")[1:].view(s.shape).copy_(s)  # noqa: E731
    d = {k: off(v) for k, v in t.items()}
    out = {k: off(torch.empty(n, D, dtype=dtype)) for k in ("out", "dx")} | {k: off(torch.empty(D)) for k in ("dw", "db")}
    mean, rstd = off(torch.empty(n)), off(torch.empty(n))
    L.oomb_layer_norm_fwd(d["x"], d["w"], d["b"], out["out"], eps=1e-5, mean=mean, rstd=rstd)
    ws = torch.empty(L.oomb_layer_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], out["dx"], dw=out["dw"], db=out["db"],
                          dx_out=d["dx_out"], workspace=ws)
    ref, tol = ln_reference(t, 1e-5, dtype)
    check(out, ref, tol)


def test_layer_norm_gradients_against_differences():
    t = ln_make(3, 40, FP, seed=7, through=False)
    out = ln_run(t, 1e-3)
    f = {k: None if v is None else v.to(F64) for k, v in t.items()}

    def total(x, w, b):
        c = x - x.mean(1, keepdim=True)
        y = c * torch.rsqrt((c * c).mean(1, keepdim=True) + 1e-3) * w + b
        return float((y * f["dy"]).sum())

    h = 1e-4
    for name, key, at in (("dx", "x", (1, 7)), ("dx", "x", (2, 39)), ("dw", "w", (3,)), ("db", "b", (11,))):
        args = []
        for s in (h, -h):
            m = {k: f[k].clone() for k in ("x", "w", "b")}
            m[key][at] += s
            args.append(total(m["x"], m["w"], m["b"]))
        assert abs((args[0] - args[1]) / (2 * h) - float(out[name][at])) <= 10 * h * h + 2e-5


def test_layer_norm_graph_replay_on_a_side_stream():
    n, D = 600, 1000
    t = ln_make(n, D, BF, seed=8)
    d = {k: v.cuda() for k, v in t.items()}
    out = {"out": torch.empty_like(d["x"]), "dx": torch.empty_like(d["x"]), "dw": torch.empty(D, device="cuda"),
           "db": torch.empty(D, device="cuda")}
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(L.oomb_layer_norm_workspace(n, D), dtype=torch.uint8, device="cuda")

    def step():
        L.oomb_layer_norm_fwd(d["x"], d["w"], d["b"], out["out"], mean=mean, rstd=rstd)
        L.oomb_layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], out["dx"], dw=out["dw"], db=out["db"],
                              dx_out=d["dx_out"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    t = ln_make(n, D, BF, seed=9)
    for k, v in t.items():
        d[k].copy_(v)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want = ln_run(t, 1e-5)
    for k in want:
        assert torch.equal(out[k], want[k]), k
