"""Layer norm of rows that lie far from 0 against their spread, and of constant ones, against float64 statistics of the
same values; the backward without a workspace where it needs none."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from ends_ref import U32, check, half_step
from test_gpu_embed_ln import OPS, ln_make, ln_reference

pytestmark = pytest.mark.gpu

BF, FP, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def run(t, eps=1e-5):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    n, D = t["x"].shape
    out = {k: torch.full((n, D), float("nan"), dtype=t["x"].dtype, device="cuda") for k in ("out", "dx")}
    out |= {k: torch.full((D,), float("nan"), device="cuda") for k in ("dw", "db")}
    out |= {k: torch.empty(n, device="cuda") for k in ("mean", "rstd")}
    L.oomb_layer_norm_fwd(d["x"], d["w"], d["b"], out["out"], eps=eps, mean=out["mean"], rstd=out["rstd"])
    ws = torch.empty(L.oomb_layer_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_layer_norm_bwd(d["x"], d["w"], out["mean"], out["rstd"], d["dy"], out["dx"], dw=out["dw"], db=out["db"],
                          dx_out=d["dx_out"], workspace=ws)
    return out


def near(t, eps=1e-5):
    """Values, and bounds that do not grow with the mean in their first order: the deviations from a mean that is off by
    OPS of itself are summed again, which leaves OPS of their size, and OPS^2 of the mean.  (Not in rows within 4 spreads
    of 0, the spread with eps in it, whose mean's OPS stays.)"""
    dt = t["x"].dtype
    ref, _ = ln_reference(t, eps, dt)
    f = {k: None if v is None else v.to(F64) for k, v in t.items()}
    w = torch.ones(t["x"].shape[1], dtype=F64) if f["w"] is None else f["w"]
    b = torch.zeros_like(w) if f["b"] is None else f["b"]
    mean = f["x"].mean(1, keepdim=True)
    c = f["x"] - mean
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + eps)
    xn, half = c * r, half_step(dt)
    size = c.abs().mean(1, keepdim=True)
    e_c = OPS * size + 3 * U32 * c.abs() + OPS ** 2 * mean.abs() + OPS * mean.abs() * (mean.abs() * r <= 4.01)
    e_r = 4 * OPS + (e_c * r).square().mean(1, keepdim=True)
    e_xn = e_c * r * 1.01 + e_r * xn.abs()
    tol = {"out": half * ref["out"].abs() + e_xn * w.abs() + 2 * U32 * (xn * w).abs() + U32 * b.abs()}
    dy = f["dy"]
    q = dy * w
    m0, m1 = q.mean(1, keepdim=True), (q * xn).mean(1, keepdim=True)
    v = r * (q - m0 - xn * m1)
    # (the sums run over xn from the mean as it was kept, which is off by 2^-24 of it, and are corrected by that)
    off = 2 * U32 * mean.abs() * r
    e_m0 = OPS * q.abs().mean(1, keepdim=True)
    e_m1 = (q.abs() * e_xn).mean(1, keepdim=True) + OPS * (q.abs() * (xn.abs() + off)).mean(1, keepdim=True)
    tol["dx"] = (half + 2 * U32) * ref["dx"].abs() + e_r * v.abs() + r * (
        e_m0 + xn.abs() * e_m1 + e_xn * m1.abs() + 4 * U32 * (q.abs() + m0.abs() + (xn * m1).abs()))
    n = dy.shape[0]
    tol["dw"] = (dy.abs() * e_xn).sum(0) + (2 * n + 32) * U32 * (dy.abs() * (xn.abs() + off)).sum(0)
    tol["db"] = (n + 32) * U32 * dy.abs().sum(0)
    ref["mean"], ref["rstd"] = mean[:, 0], r[:, 0]
    tol["mean"] = (U32 * mean.abs() + OPS * size + OPS ** 2 * mean.abs() + OPS * mean.abs() * (mean.abs() * r <= 4.01))[:, 0]
    tol["rstd"] = (e_r * r)[:, 0]
    return ref, tol


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("far", [1e2, 1e3, 1e4, 1e5])
@pytest.mark.parametrize("n,D", [(9, 1024), (40, 3584), (400, 1001), (5, 16384), (33, 9001), (700, 64), (3, 7)])
def test_rows_far_from_zero(dtype, far, n, D):
    t = ln_make(n, D, FP, seed=D)
    sign = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)[:, None]
    t["x"] = t["x"] / 3 + far * sign * (1 + torch.arange(n)[:, None] / n)
    t = {k: v.to(dtype) if k in ("x", "dy", "dx_out") else v for k, v in t.items()}
    check(run(t), *near(t))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("value", [1000.1, -33333.3, 1e-3, 0.0])
@pytest.mark.parametrize("n,D", [(4, 100), (20, 3584), (3, 9001)])
def test_constant_rows(dtype, value, n, D):
    """No spread: the output is the bias."""
    t = ln_make(n, D, dtype, seed=2)
    t["x"][:] = value
    check(run(t), *near(t))


def test_rows_of_both_kinds_by_their_blocks():
    """Near and far rows one after another, more than there are blocks."""
    t = ln_make(3000, 520, FP, seed=8, through=False)
    t["x"][::3] += 2e4
    check(run(t), *near(t))


@pytest.mark.parametrize("n,D", [(5, 64), (16, 1000), (17, 1000), (700, 3584)])
def test_backward_without_parameter_gradients_needs_no_workspace(n, D):
    t = ln_make(n, D, BF, seed=n)
    d = {k: v.cuda() for k, v in t.items()}
    want = run(t)
    dx = torch.full_like(d["x"], float("nan"))
    L.oomb_layer_norm_bwd(d["x"], d["w"], want["mean"], want["rstd"], d["dy"], dx, dx_out=d["dx_out"])
    assert torch.equal(dx, want["dx"])
    with pytest.raises(L.OombError, match="ERR_WORKSPACE"):
        L.oomb_layer_norm_bwd(d["x"], d["w"], want["mean"], want["rstd"], d["dy"], dx, dw=torch.empty(D, device="cuda"))
