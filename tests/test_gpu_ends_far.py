"""Tensors of more than 2^31 elements at a model's two ends: the last rows count, on every way to them."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from ends_ref import check, half_step, head_reference
from test_gpu_head_loss import word

pytestmark = pytest.mark.gpu

BF, FP, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


@pytest.mark.parametrize("D", [3600, 3601])
def test_a_long_vocabulary_on_the_tensor_cores(D):
    """W in place and through the workspace; its rows are 0 but for the last 64, whose neighbours share one logit."""
    V, n = 600_001, 40
    room(40)
    g = torch.Generator().manual_seed(0)
    w = torch.zeros(V, D, dtype=BF, device="cuda")
    tail = (torch.randn(64, D, generator=g) * 0.03).to(BF)
    w[-64:] = tail.cuda()
    x, d = torch.randn(n, D, generator=g).to(BF), 0.5 + torch.rand(n, generator=g)
    t = torch.randint(V - 64, V, (n,), generator=g)
    t[0], t[1], t[2] = V - 1, V - 64, 5
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, BF, True), dtype=torch.uint8, device="cuda")
    loss, lse, err = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), word()
    xs, ts, dx, dw = x.cuda(), t.cuda(), torch.empty(n, D, dtype=BF, device="cuda"), torch.empty_like(w)
    L.oomb_head_loss_fwd(xs, w, ts, loss, lse, ws, err)
    L.oomb_head_loss_bwd(xs, w, ts, lse, dx, dw, ws, err, d_loss=d.cuda())
    assert L.oomb_word_check(err) == 0
    z = torch.cat([torch.zeros(n, 1, dtype=F64), x.to(F64) @ tail.to(F64).t()], 1)
    more = z.clone()
    more[:, 0] = torch.log(torch.tensor(float(V - 64), dtype=F64))
    want = torch.logsumexp(more, 1)
    at = torch.where(t < V - 64, torch.zeros_like(t), t - (V - 64) + 1)
    # a logit: (D + 32) 2^-24 of its products' magnitudes; the sum over V / 128 parts of 128 columns: 600 + V / 64 roundings
    e = (D + 32) * 2.0 ** -24 * (x.to(F64).abs() @ tail.to(F64).abs().t()).amax(1) + (600 + V / 64) * 2.0 ** -24 + 1e-5
    assert ((lse.cpu().to(F64) - want).abs() <= e).all()
    assert ((loss.cpu().to(F64) - (want - z[torch.arange(n), at])).abs() <= 2 * e).all()
    q = torch.exp(z[:, 1:] - want[:, None])
    q[torch.arange(n)[at > 0], at[at > 0] - 1] -= 1
    q = q * d[:, None]
    rel = 2 * half_step(BF) + 4 * e.max()  # dz's rounding and the output's, and the exponents'
    for got, a, b in ((dw[-64:], q.t(), x.to(F64)), (dx, q, tail.to(F64))):
        assert ((got.cpu().to(F64) - a @ b).abs() <= rel * (a.abs() @ b.abs()) + 1e-6).all()
    five = (torch.exp(-want)[2] - 1) * d[2] * x[2].to(F64)
    others = (torch.exp(-want) * d) @ x.to(F64) - torch.exp(-want)[2] * d[2] * x[2].to(F64)
    assert ((dw[5].cpu().to(F64) - five - others).abs() <= rel * (five.abs() + 1e-4)).all()


def test_many_rows_of_a_short_vocabulary():
    """x, dx and the sums of dx past 2^31 elements: rows of zeros, but for some at both ends."""
    n, V, D = 600_001, 64, 3600
    room(60)
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(V, D, generator=g) / 60).to(BF)
    some = torch.cat([torch.arange(20), torch.arange(n - 300, n)])
    x, t = torch.zeros(n, D, dtype=BF, device="cuda"), torch.full((n,), 3, device="cuda")
    part, pt = torch.randn(320, D, generator=g).to(BF), torch.randint(0, V, (320,), generator=g)
    x[some.cuda()], t[some.cuda()] = part.cuda(), pt.cuda()
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, BF, True), dtype=torch.uint8, device="cuda")
    loss, lse, err = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), word()
    dx, dw = torch.empty_like(x), torch.empty(V, D, device="cuda")
    L.oomb_head_loss_fwd(x, w.cuda(), t, loss, lse, ws, err)
    L.oomb_head_loss_bwd(x, w.cuda(), t, lse, dx, dw, ws, err)
    assert L.oomb_word_check(err) == 0
    ref, tol = head_reference(part, w, pt, dw_dtype=FP)
    pick = some.cuda()
    check({"loss": loss[pick], "lse": lse[pick], "dx": dx[pick], "dw": dw}, ref, tol)  # rows of zeros add nothing to dw
    ref, tol = head_reference(torch.zeros(1, D, dtype=BF), w, torch.tensor([3]))
    for i in (20, n // 2, n - 301):
        check({"loss": loss[i:i + 1], "dx": dx[i:i + 1]}, ref, tol, ("loss", "dx"))


def test_layer_norm_of_many_rows():
    n, D = 600_001, 3600
    room(40)
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(n, D, generator=g, device="cuda", dtype=BF)
    dy = torch.zeros_like(x)
    some = torch.cat([torch.arange(7), torch.arange(n - 300, n)]).cuda()
    dy[some] = torch.randn(some.numel(), D, generator=g, device="cuda", dtype=BF)
    w, b = 1 + 0.3 * torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")

    def both(x, dy):
        out, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(x.shape[0], device="cuda"), torch.empty(x.shape[0], device="cuda")
        dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        L.oomb_layer_norm_fwd(x, w, b, out, mean=mean, rstd=rstd)
        ws = torch.empty(L.oomb_layer_norm_workspace(x.shape[0], D), dtype=torch.uint8, device="cuda")
        L.oomb_layer_norm_bwd(x, w, mean, rstd, dy, dx, dw=dw, db=db, workspace=ws)
        return out, dx, mean, rstd, dw, db

    far, near = both(x, dy), both(x[some].contiguous(), dy[some].contiguous())
    for a, c in zip(far[:4], near[:4]):  # a row's values are its own
        assert torch.equal(a[some], c)
    xn = (x[some].to(F64) - near[2][:, None]) * near[3][:, None]
    for a, c, m in ((far[4], near[4], (dy[some].to(F64) * xn).abs().sum(0)), (far[5], near[5], dy[some].to(F64).abs().sum(0))):
        assert ((a - c).to(F64).abs() <= 2 * (307 + 32) * 2.0 ** -24 * m).all()  # the same terms in another order


@pytest.mark.parametrize("D", [3600, 3601])
def test_embeddings_of_many_rows(D):
    n, V = 600_001, 50
    room(40)
    g = torch.Generator("cuda").manual_seed(3)
    t = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    t[:5], t[-300:] = torch.arange(5, device="cuda"), torch.randint(0, V, (300,), generator=g, device="cuda")
    t[5:n - 300:2] = 7
    tab = torch.randn(V, D, generator=g, device="cuda", dtype=BF)
    out, err = torch.full((n, D), float("nan"), dtype=BF, device="cuda"), word()
    L.oomb_embed_fwd(t, tab, out, err)
    for i in (0, 5, 6, n // 2, n - 301, n - 300, n - 1):
        assert torch.equal(out[i], tab[t[i]] if t[i] >= 0 else torch.zeros_like(tab[0])), i
    d = out
    d.zero_()
    d[-300:] = torch.randn(300, D, generator=g, device="cuda", dtype=BF)
    grad = torch.zeros(V, D, device="cuda")
    ws = torch.empty(L.oomb_embed_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_embed_bwd(t, d, grad, ws, err)
    assert L.oomb_word_check(err) == 0
    want = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, t[-300:], d[-300:].to(F64))
    size = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, t[-300:], d[-300:].to(F64).abs())
    assert ((grad.to(F64) - want).abs() <= 316 * 2.0 ** -24 * size).all()
