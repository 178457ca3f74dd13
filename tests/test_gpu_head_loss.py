"""Cross entropy over a vocabulary without keeping the logits, on the GPU against float64."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from ends_ref import check, head_reference

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(n, V, D, dtype, seed=0, masked=0.0, lean=4.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) * (1.2 / D ** 0.5)).to(dtype)
    t = torch.randint(0, V, (n,), generator=g)
    x = (torch.randn(n, D, generator=g) + lean * w[t].float() / w[t].float().norm(dim=1, keepdim=True)).to(dtype)
    t = torch.where(torch.rand(n, generator=g) < masked, torch.full_like(t, -100), t)
    return x, w, t, 0.25 + torch.rand(n, generator=g)


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def run(x, w, t, cap=0.0, d_loss=None, scale=1.0, dw_dtype=None, accumulate=False, base=None, dx=True, dw=True,
        ws=None, stream=None):
    x, w, t = x.cuda(), w.cuda(), t.cuda()
    d_loss = None if d_loss is None else d_loss.cuda()
    n, D = x.shape
    V = w.shape[0]
    nan = lambda *s, dt=FP: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out = {"loss": nan(n), "lse": nan(n), "dx": nan(n, D, dt=x.dtype) if dx else None, "dw": None}
    if dw:
        out["dw"] = nan(V, D, dt=dw_dtype or w.dtype) if base is None else base.cuda()
    err = word()
    if ws is None:
        ws = torch.full((L.oomb_head_loss_workspace(n, D, V, x.dtype, True),), 255, dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(x, w, t, out["loss"], out["lse"], ws, err, softcap=cap)
    L.oomb_head_loss_bwd(x, w, t, out["lse"], out["dx"], out["dw"], ws, err, d_loss=d_loss, scale=scale, softcap=cap,
                         accumulate=accumulate)
    assert L.oomb_word_check(err) == 0
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (1, 1, 8), (1, 100, 64), (2, 3, 7), (33, 1000, 128), (5, 130, 9),
                                   (64, 64, 64), (127, 255, 72), (128, 256, 64), (129, 257, 136), (257, 513, 1000),
                                   (300, 4099, 65), (511, 300, 264), (1, 20001, 256), (700, 129, 2048)])
def test_head_matches(dtype, n, V, D):
    x, w, t, _ = make(n, V, D, dtype, seed=n + V)
    ref, tol = head_reference(x, w, t)
    check(run(x, w, t), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap", [0.0, 30.0, 2.0])
@pytest.mark.parametrize("masked", [0.0, 0.6])
def test_caps_masks_weights_and_scale(dtype, cap, masked):
    x, w, t, g = make(203, 1111, 96, dtype, seed=7, masked=masked)
    g[::5] = 0.0
    g[1::7] *= -3.0
    kw = dict(cap=cap, d_loss=g, scale=1.0 / 203)
    ref, tol = head_reference(x, w, t, **kw)
    check(run(x, w, t, **kw), ref, tol)


def test_several_pieces_of_the_vocabulary():
    """Pieces that dz's share of the workspace sets (many rows) and that staged rows of W set (wide fp32)."""
    for n, V, D, dt in ((70, 40961, 64, BF), (70, 40961, 72, FP), (4600, 33000, 64, BF), (1500, 33001, 40, FP),
                        (300, 3000, 20000, FP)):
        x, w, t, g = make(n, V, D, dt, seed=3, masked=0.2)
        kw = dict(d_loss=g, scale=0.5)
        ref, tol = head_reference(x, w, t, **kw)
        check(run(x, w, t, **kw), ref, tol)


@pytest.mark.parametrize("n,V,dtype", [(16500, 16700, BF), (9500, 9700, FP)])
def test_several_pieces_for_many_rows_of_which_few_count(n, V, dtype):
    """dz has room for every row; those without a target neither add to the gradients nor are read."""
    x, w, t, g = make(n, V, 72, dtype, seed=4, masked=0.96)
    has = t >= 0
    kw = dict(cap=20.0, d_loss=g, scale=0.5)
    x[~has] = float("nan")
    out = run(x, w, t, **kw)
    for k in ("loss", "lse", "dx"):
        assert (out[k].cpu()[~has] == 0).all(), k
        out[k] = out[k].cpu()[has]
    ref, tol = head_reference(x[has], w, t[has], cap=20.0, d_loss=g[has], scale=0.5)
    check(out, ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [150, 24])
def test_rows_without_a_target(dtype, n):
    """No row has one; or only a few do, and the others hold infinities and NaN."""
    x, w, t, _ = make(n, 300, 64, dtype, seed=1)
    none = torch.full_like(t, -1)
    out = run(x, w, none)
    for k in ("loss", "lse", "dx", "dw"):
        assert (out[k] == 0).all(), k
    few = none.clone()
    few[[3, n * 5 // 6, n - 2, n - 1]] = t[[3, n * 5 // 6, n - 2, n - 1]]
    bad = x.clone()
    bad[few < 0] = float("nan")
    bad[0, 0], bad[1, 1] = float("inf"), float("-inf")
    ref, tol = head_reference(x, w, few)
    check(run(bad, w, few), ref, tol)


def test_a_target_behind_the_vocabulary_is_told():
    x, w, t, _ = make(40, 100, 64, BF, seed=2)
    bad = t.clone()
    bad[7], bad[39] = 100, 2 ** 40
    plain = torch.where(bad >= 100, torch.full_like(bad, -1), bad)
    good = run(x, w, plain)
    out = {k: torch.empty_like(v) for k, v in good.items()}
    err, xs, ws_, ts = word(), x.cuda(), w.cuda(), bad.cuda()
    ws = torch.empty(L.oomb_head_loss_workspace(40, 64, 100, BF, True), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(xs, ws_, ts, out["loss"], out["lse"], ws, err)
    with pytest.raises(L.OombError, match="0x20"):
        L.oomb_word_check(err)
    L.oomb_head_loss_bwd(xs, ws_, ts, out["lse"], out["dx"], out["dw"], ws, err)
    with pytest.raises(L.OombError, match="0x20"):
        L.oomb_word_check(err)
    assert L.oomb_word_check(err) == 0
    for k in good:
        assert torch.equal(out[k], good[k]), k


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap", [3e2, 1e5, 1e30, 1e-3, 1e-30])
@pytest.mark.parametrize("n", [20, 100])
def test_caps_far_above_and_below_the_logits(dtype, cap, n):
    """A cap far above the logits leaves them as they are; under one far below they are all alike."""
    x, w, t, _ = make(n, 500, 72, dtype, seed=17)
    ref, tol = head_reference(x, w, t, cap=cap)
    check(run(x, w, t, cap=cap), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_the_widest_rows(dtype):
    x, w, t, g = make(3, 5, 65536, dtype, seed=19)
    ref, tol = head_reference(x, w, t, d_loss=g)
    check(run(x, w, t, d_loss=g), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [140, 20])
def test_one_gradient_alone_and_fp32_weights_gradient(dtype, n):
    x, w, t, g = make(n, 700, 88, dtype, seed=5, masked=0.1)
    both = run(x, w, t, d_loss=g)
    assert torch.equal(run(x, w, t, d_loss=g, dw=False)["dx"], both["dx"])
    assert torch.equal(run(x, w, t, d_loss=g, dx=False)["dw"], both["dw"])
    out = run(x, w, t, d_loss=g, dw_dtype=FP)
    ref, tol = head_reference(x, w, t, d_loss=g, dw_dtype=FP)
    check(out, ref, tol)
    assert torch.equal(out["dw"].to(dtype), both["dw"])
    base = torch.randn(700, 88, generator=torch.Generator().manual_seed(8))
    add = run(x, w, t, d_loss=g, accumulate=True, base=base)["dw"].cpu()
    slack = 2 ** -23 * (base.abs() + out["dw"].cpu().abs())
    assert ((add.double() - (base.double() + out["dw"].cpu().double())).abs() <= slack).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,V,D", [(140, 700, 89), (140, 31000, 261), (140, 31000, 264), (600, 31001, 33)])
def test_gradients_added_in_rows_of_every_alignment(dtype, n, V, D):
    x, w, t, g = make(n, V, D, dtype, seed=6, masked=0.1)
    plain = run(x, w, t, d_loss=g, dw_dtype=FP)["dw"].cpu()
    base = torch.randn(V, D, generator=torch.Generator().manual_seed(9))
    add = run(x, w, t, d_loss=g, accumulate=True, base=base)["dw"].cpu()
    slack = 2 ** -23 * (base.abs() + plain.abs())  # a rounding of each
    assert ((add.double() - (base.double() + plain.double())).abs() <= slack).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [300, 7])
def test_the_same_bits_on_every_run(dtype, n):
    x, w, t, g = make(n, 5000, 200, dtype, seed=9, masked=0.3)
    a, b = run(x, w, t, cap=30.0, d_loss=g), run(x, w, t, cap=30.0, d_loss=g)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [60, 140])
def test_tensors_off_16_bytes(dtype, n):
    x, w, t, g = make(n, 333, 64, dtype, seed=11)
    want = run(x, w, t, d_loss=g)
    off = lambda s, dt: torch.empty(s.numel() + 1, dtype=dt, device="cuda")[1:].view(s.shape)  # noqa: E731
    xo, wo = off(x, dtype).copy_(x), off(w, dtype).copy_(w)
    out = {"loss": off(t, FP), "lse": off(t, FP), "dx": off(x, dtype), "dw": off(w, dtype)}
    go, to = off(g, FP).copy_(g), t.cuda()
    err = word()
    ws = torch.empty(L.oomb_head_loss_workspace(n, 64, 333, dtype, True), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(xo, wo, to, out["loss"], out["lse"], ws, err)
    L.oomb_head_loss_bwd(xo, wo, to, out["lse"], out["dx"], out["dw"], ws, err, d_loss=go)
    assert L.oomb_word_check(err) == 0
    check(out, *head_reference(x, w, t, d_loss=g))
    for k in want:  # few rows: a thread has other columns, whose products are added in another order
        assert n < 64 or torch.equal(out[k], want[k]), k


def test_a_wide_projection_off_16_bytes():
    """bf16 rows that are read through the workspace, in two pieces."""
    x, w, t, g = make(20, 9000, 2048, BF, seed=13, masked=0.2)
    want = run(x, w, t, d_loss=g)
    wo = torch.empty(w.numel() + 1, dtype=BF, device="cuda")[1:].view(w.shape).copy_(w)
    out = {k: torch.empty_like(v) for k, v in want.items()}
    xs, ts, gs, err = x.cuda(), t.cuda(), g.cuda(), word()
    ws = torch.empty(L.oomb_head_loss_workspace(20, 2048, 9000, BF, True), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(xs, wo, ts, out["loss"], out["lse"], ws, err)
    L.oomb_head_loss_bwd(xs, wo, ts, out["lse"], out["dx"], out["dw"], ws, err, d_loss=gs)
    assert L.oomb_word_check(err) == 0
    ref, tol = head_reference(x, w, t, d_loss=g)
    check(out, ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,V,D", [(9, 700, 3000), (40, 300, 517), (64, 257, 1000), (65, 257, 1000), (100, 9800, 72),
                                   (200, 20, 3), (2000, 40, 65), (257, 12000, 130), (8, 1842, 3840), (7, 13710, 108),
                                   (3, 1, 20), (63, 2, 9000), (2, 5, 30000)])
def test_the_ways_of_few_rows_and_few_tiles(dtype, n, V, D):
    """On both sides of the rules that choose the kernels, with targets missing and at the ends."""
    x, w, t, g = make(n, V, D, dtype, seed=n + D, masked=0.25)
    t[0], t[-1] = 0, V - 1
    kw = dict(d_loss=g, cap=20.0, scale=2.0)
    ref, tol = head_reference(x, w, t, **kw)
    check(run(x, w, t, **kw), ref, tol)
    out = run(x, w, t, dw_dtype=FP, **kw)
    ref, tol = head_reference(x, w, t, dw_dtype=FP, **kw)
    check(out, ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,V,D", [(8, 9000, 520), (16, 9000, 520), (17, 9000, 520), (24, 3000, 40), (64, 1000, 1000),
                                   (65, 1000, 100)])
def test_both_sides_of_the_rows_that_count_as_few(dtype, n, V, D):
    x, w, t, g = make(n, V, D, dtype, seed=V, masked=0.1)
    kw = dict(cap=9.0, d_loss=g, scale=0.1)
    ref, tol = head_reference(x, w, t, **kw)
    check(run(x, w, t, **kw), ref, tol)


def test_large_and_far_logits():
    """Logits of thousands in both signs: the loss of a sure row is the distance, and nothing overflows."""
    D, V = 64, 600
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(90, D, generator=g) * 60).to(BF)
    w = (torch.randn(V, D, generator=g) * 8).to(BF)
    t = torch.randint(0, V, (90,), generator=g)
    for cap in (0.0, 50.0):
        ref, tol = head_reference(x, w, t, cap=cap)
        check(run(x, w, t, cap=cap), ref, tol)


def test_two_calls_at_once_on_two_streams():
    """Each with a workspace of its own, one of them for few rows; the error word is shared."""
    sets = [make(n, 3000, 256, BF, seed=n, masked=0.2) for n in (500, 5, 300)]
    want = [run(x, w, t, d_loss=g) for x, w, t, g in sets]
    err, jobs = word(), []
    for x, w, t, g in sets:
        x, w, t, g = x.cuda(), w.cuda(), t.cuda(), g.cuda()
        ws = torch.empty(L.oomb_head_loss_workspace(x.shape[0], 256, 3000, BF, True), dtype=torch.uint8, device="cuda")
        out = {"loss": torch.empty_like(g), "lse": torch.empty_like(g), "dx": torch.empty_like(x), "dw": torch.empty_like(w)}
        jobs.append((torch.cuda.Stream(), x, w, t, g, ws, out))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, x, w, t, g, ws, out in jobs:
            L.oomb_head_loss_fwd(x, w, t, out["loss"], out["lse"], ws, err, stream=s)
            L.oomb_head_loss_bwd(x, w, t, out["lse"], out["dx"], out["dw"], ws, err, d_loss=g, stream=s)
    torch.cuda.synchronize()
    assert L.oomb_word_check(err) == 0
    for job, ref in zip(jobs, want):
        for k in ref:
            assert torch.equal(job[6][k], ref[k]), k


def test_gradients_against_differences():
    x, w, t, g = make(4, 30, 16, FP, seed=6)
    kw = dict(cap=3.0, d_loss=g, scale=0.7)
    out = run(x, w, t, **kw)

    def total(x, w):
        return float((head_reference(x, w, t, cap=3.0, grads=False)[0]["loss"] * g.double()).sum()) * 0.7

    h = 1e-4
    for name, v in (("dx", x), ("dw", w)):
        for at in [(0, 0), (1, 5), (3, 15), (2, 9)]:
            up, dn = v.double().clone(), v.double().clone()
            up[at] += h
            dn[at] -= h
            pair = [(u, w.double()) if name == "dx" else (x.double(), u) for u in (up, dn)]
            slope = (total(*pair[0]) - total(*pair[1])) / (2 * h)
            # central differences: h^2 times a third derivative below 10, and fp32's share of the gradient
            assert abs(float(out[name][at]) - slope) <= 10 * h * h + 2e-5


def test_workspace_of_a_longer_call_and_nothing_behind_it():
    sizes = [L.oomb_head_loss_workspace(n, 200, 3000, BF, b) for b in (False, True) for n in (1, 2, 127, 500, 9000)]
    assert sizes[:5] == sorted(sizes[:5]) and sizes[5:] == sorted(sizes[5:])
    assert all(a <= b for a, b in zip(sizes[:5], sizes[5:]))
    for n, dt in ((77, BF), (77, FP), (300, BF)):
        x, w, t, _ = make(n, 3000, 200, dt, seed=n)
        size = L.oomb_head_loss_workspace(n, 200, 3000, dt, True)
        ws = torch.full((size + 4096,), 171, dtype=torch.uint8, device="cuda")
        ref, tol = head_reference(x, w, t)
        check(run(x, w, t, ws=ws[:size]), ref, tol)
        assert (ws[size:] == 171).all()
        big = torch.full((L.oomb_head_loss_workspace(1000, 200, 3000, dt, True),), 9, dtype=torch.uint8, device="cuda")
        check(run(x, w, t, ws=big), ref, tol)


@pytest.mark.parametrize("n", [150, 6])
def test_graph_replays_on_a_side_stream_with_new_data(n):
    V, D = 2000, 128
    x, w, t, g = make(n, V, D, BF, seed=1, masked=0.2)
    xs, wsd, ts, gs = x.cuda(), w.cuda(), t.cuda(), g.cuda()
    out = {"loss": torch.empty(n, device="cuda"), "lse": torch.empty(n, device="cuda"), "dx": torch.empty_like(xs),
           "dw": torch.empty_like(wsd)}
    err = word()
    space = torch.empty(L.oomb_head_loss_workspace(n, D, V, BF, True), dtype=torch.uint8, device="cuda")

    def step():
        L.oomb_head_loss_fwd(xs, wsd, ts, out["loss"], out["lse"], space, err)
        L.oomb_head_loss_bwd(xs, wsd, ts, out["lse"], out["dx"], out["dw"], space, err, d_loss=gs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (2, 3):
        x, w, t, g = make(n, V, D, BF, seed=seed, masked=0.1 * seed)
        for a, b in ((xs, x), (wsd, w), (ts, t), (gs, g)):
            a.copy_(b)
        torch.cuda.synchronize()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        want = run(x, w, t, d_loss=g)
        for k in want:
            assert torch.equal(out[k], want[k]), k
    assert L.oomb_word_check(err) == 0


def test_offsets_past_32_bits():
    """More than 2^31 elements of W: the last rows of the vocabulary count."""
    V, D, n = 600_001, 3600, 3
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    w = torch.zeros(V, D, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(0)
    tail = (torch.randn(64, D, generator=g) * 0.3).to(BF)
    w[-64:] = tail.cuda()
    x = torch.randn(n, D, generator=g).to(BF)
    t = torch.tensor([V - 1, V - 64, 5])
    out = run(x, w, t)
    # logits of the zero rows are 0: the distribution is that of the tail and V - 64 zeros
    z = torch.cat([torch.zeros(n, 1, dtype=torch.float64), x.double() @ tail.double().t()], 1)
    z[:, 0] += torch.log(torch.tensor(float(V - 64), dtype=torch.float64))
    lse = torch.logsumexp(z, 1)
    loss = lse - torch.stack([z[0, 64], z[1, 1], torch.zeros((), dtype=torch.float64)])
    assert (out["lse"].cpu().double() - lse).abs().max() < 2e-3
    assert (out["loss"].cpu().double() - loss).abs().max() < 2e-3
    p = torch.exp(torch.cat([torch.zeros(n, 1, dtype=torch.float64), z[:, 1:]], 1) - lse[:, None])
    q = p[:, 1:].clone()
    q[0, 63] -= 1
    q[1, 0] -= 1
    dw = q.t() @ x.double()
    bound = 2.0 ** -7 * (q.abs().t() @ x.double().abs()) + 1e-6
    assert ((out["dw"][-64:].cpu().double() - dw).abs() <= bound).all()
    dx = q @ tail.double()
    bound = 2.0 ** -7 * (q.abs() @ tail.double().abs()) + 1e-6
    assert ((out["dx"].cpu().double() - dx).abs() <= bound).all()
