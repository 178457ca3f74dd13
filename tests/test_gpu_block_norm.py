"""The norms around a block with its gate and residual scale, on the GPU against float64."""
import pytest
import torch

import paged_sparse_attention_gb300 as L

pytestmark = pytest.mark.gpu

BF, FP, F64 = torch.bfloat16, torch.float32, torch.float64
U32 = 2.0 ** -24
# fp32 roundings on the way to an element: at most 32 terms a thread (16384 / 512), 10 steps of
# the block's sum, and a dozen products
OPS = 64 * U32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(n, D, dtype, gate, post, pre=True, block=True, dx_out=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = {"x": torch.randn(n, D, generator=g).mul(3).to(dtype)}
    t["y"] = torch.randn(n, D, generator=g).to(dtype) if block else None
    t["w_post"] = 1 + 0.3 * torch.randn(D, generator=g) if post and block else None
    t["w_pre"] = 1 + 0.3 * torch.randn(D, generator=g) if pre else None
    t["gate"] = None
    if gate == "channel" and block:
        t["gate"] = torch.randn(D, generator=g)
    if gate == "token" and block:
        t["gate"] = torch.randn(n, D, generator=g).to(dtype)
    t["du"] = torch.randn(n, D, generator=g).to(dtype) if pre else None
    t["dx_out"] = torch.randn(n, D, generator=g).to(dtype) if dx_out or not pre else None
    return t


def reference(t, a, eps, dtype):
    """Values in float64 and bounds: one rounding to the output's type, and OPS on the
    magnitudes of the terms that an output is the sum of."""
    half = torch.finfo(dtype).eps / 2
    f = {k: None if v is None else v.to(F64) for k, v in t.items()}
    x, y = f["x"], f["y"]
    n, D = x.shape
    ref, tol = {}, {}
    xo, mag = x, x.abs()
    if y is not None:
        yn, z = y, y
        r_post = torch.ones(n, 1, dtype=F64)
        if f["w_post"] is not None:
            r_post = torch.rsqrt(y.pow(2).mean(1, keepdim=True) + eps)
            yn = y * r_post
            z = yn * f["w_post"]
        g = torch.ones(D, dtype=F64) if f["gate"] is None else f["gate"]
        xo = x + a * g * z
        mag = x.abs() + (a * g * z).abs()
    ref["x_out"], tol["x_out"] = xo, half * xo.abs() + OPS * mag
    dx = torch.zeros_like(x) if f["dx_out"] is None else f["dx_out"]
    dmag = dx.abs()
    if f["w_pre"] is not None:
        r = torch.rsqrt(xo.pow(2).mean(1, keepdim=True) + eps)
        xn = xo * r
        e_xn = OPS * (mag * r + xn.abs())  # of x_out r_pre before it is rounded
        ref["u"] = xn * f["w_pre"]
        tol["u"] = half * ref["u"].abs() + 2 * e_xn * f["w_pre"].abs()
        q = f["du"] * f["w_pre"]
        m = (q * xn).mean(1, keepdim=True)
        e_m = ((q.abs() * e_xn).mean(1, keepdim=True) + OPS * (q * xn).abs().mean(1, keepdim=True))
        dx = dx + r * (q - xn * m)
        dmag = dmag + r * (q.abs() + (xn * m).abs()) + r * (e_xn * m.abs() + xn.abs() * e_m) / OPS
        ref["dw_pre"] = (f["du"] * xn).sum(0)
        tol["dw_pre"] = (f["du"].abs() * e_xn).sum(0) + (n + 32) * U32 * (f["du"] * xn).abs().sum(0)
    ref["dx"], tol["dx"] = dx, half * dx.abs() + 2 * OPS * dmag
    if y is not None:
        e_dx = 2 * OPS * dmag
        dgz = a * dx
        dz = dgz * g
        if f["gate"] is not None:
            v, e = dgz * z, abs(a) * e_dx * z.abs() + OPS * (dgz * z).abs()
            if f["gate"].dim() == 2:
                ref["dgate"], tol["dgate"] = v, e + half * v.abs()
            else:
                ref["dgate"], tol["dgate"] = v.sum(0), e.sum(0) + (n + 32) * U32 * v.abs().sum(0)
        e_dz = abs(a) * e_dx * g.abs() + OPS * dz.abs()
        dy, e_dy = dz, e_dz
        if f["w_post"] is not None:
            v = dz * yn
            ref["dw_post"] = v.sum(0)
            tol["dw_post"] = (e_dz * yn.abs() + OPS * v.abs()).sum(0) + (n + 32) * U32 * v.abs().sum(0)
            q, e_q = dz * f["w_post"], e_dz * f["w_post"].abs()
            m = (q * yn).mean(1, keepdim=True)
            e_m = (e_q * yn.abs()).mean(1, keepdim=True) + OPS * (q * yn).abs().mean(1, keepdim=True)
            dy = r_post * (q - yn * m)
            e_dy = r_post * (e_q + yn.abs() * e_m + OPS * (q.abs() + (yn * m).abs()))
        ref["dy"], tol["dy"] = dy, half * dy.abs() + 2 * e_dy
    return ref, tol


def run(t, a, eps, dtype, accumulate=False, base=None):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    n, D = t["x"].shape
    new = lambda: torch.full((n, D), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    vec = lambda: torch.full((D,), float("nan") if base is None else base, device="cuda")  # noqa: E731
    par = dict(w_pre=d["w_pre"], w_post=d["w_post"], gate=d["gate"], res_scale=a)
    out = {"x_out": new()}
    out["u"] = new() if d["w_pre"] is not None else None
    r_pre = torch.empty(n, device="cuda") if d["w_pre"] is not None else None
    r_post = torch.empty(n, device="cuda") if d["w_post"] is not None else None
    L.oomb_block_norm_fwd(d["x"], d["y"], out["x_out"], out["u"], eps=eps, rstd_pre=r_pre, rstd_post=r_post, **par)
    out["dx"] = new()
    out["dy"] = new() if d["y"] is not None else None
    out["dw_pre"] = vec() if d["w_pre"] is not None else None
    out["dw_post"] = vec() if d["w_post"] is not None else None
    out["dgate"] = None if d["gate"] is None else vec() if d["gate"].dim() == 1 else new()
    ws = torch.empty(L.oomb_block_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_block_norm_bwd(d["x"], d["y"], out["dx"], out["dy"], du=d["du"], dx_out=d["dx_out"], rstd_pre=r_pre,
                          rstd_post=r_post, dw_pre=out["dw_pre"], dw_post=out["dw_post"], dgate=out["dgate"],
                          accumulate=accumulate, workspace=ws, **par)
    return out


def compare(out, ref, tol, base=0.0):
    for k, r in ref.items():
        shift = base if r.dim() == 1 else 0.0
        g = out[k].cpu().to(F64)
        assert torch.isfinite(g).all(), k
        slack = tol[k] + (2 * U32 * (r.abs() + abs(shift)) if shift else 0.0)
        over = (g - (r + shift)).abs() - slack
        assert over.max().item() <= 0, (k, over.max().item(), slack.flatten()[over.argmax()].item())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [8, 64, 256, 1000, 1023, 3584, 4104, 8192, 9000, 16384, 1, 7])
@pytest.mark.parametrize("gate,post", [("channel", True), ("token", True), ("none", False), ("token", False)])
def test_block_norm_matches(dtype, D, gate, post):
    n = 37 if D < 4000 else 5
    t = make(n, D, dtype, gate, post, seed=D)
    ref, tol = reference(t, 0.7, 1e-6, dtype)
    compare(run(t, 0.7, 1e-6, dtype), ref, tol)


@pytest.mark.parametrize("n", [1, 2, 303, 1501])
def test_rows(n):
    """One row, fewer and more rows than there are thread blocks."""
    t = make(n, 200, BF, "channel", True, seed=n)
    ref, tol = reference(t, -1.5, 1e-5, BF)
    compare(run(t, -1.5, 1e-5, BF), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,D", [(1301, 3584), (2001, 2048), (5003, 256), (2501, 4112), (1303, 8192)])
@pytest.mark.parametrize("kw", [dict(gate="channel", post=True), dict(gate="token", post=True, dx_out=False),
                                dict(gate="none", post=False), dict(gate="none", post=False, block=False),
                                dict(gate="token", post=True, pre=False)])
def test_many_rows(dtype, n, D, kw):
    """Enough rows for each thread block to walk several."""
    t = make(n, D, dtype, seed=n, **kw)
    ref, tol = reference(t, 0.7, 1e-6, dtype)
    compare(run(t, 0.7, 1e-6, dtype), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,D", [(1301, 3577), (2001, 517), (901, 5122), (701, 8191), (1303, 132), (1501, 41), (700, 5120)])
@pytest.mark.parametrize("kw", [dict(gate="channel", post=True), dict(gate="token", post=True)])
def test_many_rows_of_any_width(dtype, n, D, kw):
    """Rows that start and end anywhere, the last one off the 16 bytes too."""
    t = make(n, D, dtype, seed=n, **kw)
    ref, tol = reference(t, 0.7, 1e-6, dtype)
    compare(run(t, 0.7, 1e-6, dtype), ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [515, 520])
def test_many_rows_in_place(dtype, D):
    """x_out over x and dx over dx_out, many rows; what stands around the tensors stays."""
    n, pad = 2601, 64
    t = make(n, D, dtype, "token", True, seed=3)
    ref, tol = reference(t, 0.5, 1e-6, dtype)
    bufs = {}

    def inside(k, v):  # with NaN around it
        bufs[k] = torch.full((n * D + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
        w = bufs[k][pad:-pad].view(n, D)
        return w if v is None else w.copy_(v)

    d = {k: inside(k, v) if v.dim() == 2 else v.cuda() for k, v in t.items()}
    x, dx, x0 = inside("x_out", t["x"]), inside("dx", t["dx_out"]), d["x"]
    u, dy, dg = inside("u", None), inside("dy", None), inside("dgate", None)
    r1, r2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dw1, dw2 = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    par = dict(w_pre=d["w_pre"], w_post=d["w_post"], gate=d["gate"], res_scale=0.5, rstd_pre=r1, rstd_post=r2)
    L.oomb_block_norm_fwd(x, d["y"], x, u, eps=1e-6, **par)
    ws = torch.empty(L.oomb_block_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_block_norm_bwd(x0, d["y"], dx, dy, du=d["du"], dx_out=dx, dgate=dg, dw_pre=dw1, dw_post=dw2, workspace=ws,
                          **par)
    compare({"x_out": x, "u": u, "dx": dx, "dy": dy, "dgate": dg, "dw_pre": dw1, "dw_post": dw2}, ref, tol)
    for k, b in bufs.items():
        assert b[:pad].isnan().all() and b[-pad:].isnan().all(), k


@pytest.mark.parametrize("D", [256, 255])
@pytest.mark.parametrize("kind", ["pre_only", "post_only", "no_residual_gradient", "gate_only"])
def test_parts_left_out(kind, D):
    kw = {"pre_only": dict(gate="none", post=False, block=False), "post_only": dict(gate="token", post=True, pre=False),
          "no_residual_gradient": dict(gate="channel", post=True, dx_out=False),
          "gate_only": dict(gate="channel", post=False, pre=False)}[kind]
    for dtype in (BF, FP):
        t = make(19, D, dtype, seed=4, **kw)
        ref, tol = reference(t, 2.0, 1e-6, dtype)
        compare(run(t, 2.0, 1e-6, dtype), ref, tol)


def test_gradients_against_differences():
    """The float64 reference's own gradients against central differences of its forward."""
    t = {k: None if v is None else v.double() for k, v in make(2, 6, FP, "token", True, seed=9).items()}
    ref, _ = reference(t, 0.7, 1e-6, FP)
    loss = lambda s: float((lambda r: (r["x_out"] * t["dx_out"]).sum() + (r["u"] * t["du"]).sum())(  # noqa: E731
        reference(s, 0.7, 1e-6, FP)[0]))
    for name, grad in (("x", "dx"), ("y", "dy"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        for i in range(0, t[name].numel(), 3):
            h = 1e-5
            up, down = t[name].clone(), t[name].clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            num = (loss({**t, name: up}) - loss({**t, name: down})) / (2 * h)
            assert abs(num - ref[grad].view(-1)[i].item()) < 1e-6 * (1 + abs(num)), (name, i)


def test_accumulate_adds_and_repeats():
    t = make(700, 512, BF, "channel", True, seed=1)
    ref, tol = reference(t, 0.7, 1e-6, BF)
    a = run(t, 0.7, 1e-6, BF, accumulate=True, base=3.0)
    compare(a, ref, tol, base=3.0)
    b = run(t, 0.7, 1e-6, BF, accumulate=True, base=3.0)
    for k in ref:
        assert torch.equal(a[k], b[k]), k  # the same bits on every run


@pytest.mark.parametrize("D", [512, 511])
def test_in_place_and_off_16_bytes(D):
    """x_out over x and dx over dx_out; rows that start off 16 bytes."""
    t = make(33, D, BF, "token", True, seed=2)
    ref, tol = reference(t, 0.5, 1e-6, BF)

    def off(v):  # the same values two bytes further on
        if v is None or v.dtype != BF:
            return None if v is None else v.cuda()
        b = torch.empty(v.numel() + 1, dtype=BF, device="cuda")
        b[1:] = v.view(-1).cuda()
        return b[1:].view(v.shape)

    d = {k: off(v) for k, v in t.items()}
    x = d["x"].clone() if D % 2 else off(t["x"])
    u, dy = torch.empty_like(x), torch.empty_like(x)
    r1, r2 = torch.empty(33, device="cuda"), torch.empty(33, device="cuda")
    par = dict(w_pre=d["w_pre"], w_post=d["w_post"], gate=d["gate"], res_scale=0.5)
    L.oomb_block_norm_fwd(x, d["y"], x, u, rstd_pre=r1, rstd_post=r2, **par)
    ws = torch.empty(L.oomb_block_norm_workspace(33, D), dtype=torch.uint8, device="cuda")
    dx = d["dx_out"]
    L.oomb_block_norm_bwd(d["x"], d["y"], dx, dy, du=d["du"], dx_out=dx, rstd_pre=r1, rstd_post=r2, workspace=ws, **par)
    compare({"x_out": x, "u": u, "dx": dx, "dy": dy}, {k: ref[k] for k in ("x_out", "u", "dx", "dy")}, tol)


def test_refusals():
    t = {k: None if v is None else v.cuda() for k, v in make(4, 64, BF, "channel", True).items()}
    o, u = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    ok = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    with pytest.raises(ValueError):  # not contiguous
        L.oomb_block_norm_fwd(t["x"].t().contiguous().t(), t["y"], o, u, **ok)
    with pytest.raises(ValueError):  # on the host
        L.oomb_block_norm_fwd(t["x"].cpu(), t["y"], o, u, **ok)
    with pytest.raises(ValueError):  # rows do not match
        L.oomb_block_norm_fwd(t["x"], t["y"][:3], o, u, **ok)
    with pytest.raises(TypeError):  # types do not match
        L.oomb_block_norm_fwd(t["x"], t["y"].float(), o, u, **ok)
    with pytest.raises(TypeError):  # parameters are fp32
        L.oomb_block_norm_fwd(t["x"], t["y"], o, u, w_pre=t["w_pre"].bfloat16())
    with pytest.raises(L.OombError):  # u without its weight
        L.oomb_block_norm_fwd(t["x"], t["y"], o, u)
    with pytest.raises(L.OombError):  # nothing to do
        L.oomb_block_norm_fwd(t["x"], None, o)
    with pytest.raises(L.OombError) as e:  # workspace too small
        L.oomb_block_norm_bwd(t["x"], t["y"], o, du=t["du"], rstd_pre=torch.ones(4, device="cuda"), w_pre=t["w_pre"],
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 9


def test_graph_replay_on_a_side_stream():
    t = {k: None if v is None else v.cuda() for k, v in make(1400, 512, BF, "token", True, seed=8).items()}
    x_out, u, dx, dy = (torch.empty_like(t["x"]) for _ in range(4))
    r = [torch.empty(1400, device="cuda") for _ in range(2)]
    dw = [torch.empty(512, device="cuda") for _ in range(2)]
    dg = torch.empty_like(t["x"])
    ws = torch.empty(L.oomb_block_norm_workspace(1400, 512), dtype=torch.uint8, device="cuda")
    par = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], res_scale=0.7, rstd_pre=r[0], rstd_post=r[1])

    def step():
        L.oomb_block_norm_fwd(t["x"], t["y"], x_out, u, **par)
        L.oomb_block_norm_bwd(t["x"], t["y"], dx, dy, du=t["du"], dx_out=t["dx_out"], dw_pre=dw[0], dw_post=dw[1],
                              dgate=dg, workspace=ws, **par)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = [v.clone() for v in (x_out, u, dx, dy, *dw, dg)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for v in (x_out, u, dx, dy, *dw, dg):
        v.zero_()
    g.replay()
    for a, b in zip(first, (x_out, u, dx, dy, *dw, dg)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last rows."""
    n, D, last = 600500, 3584, 64
    small = make(last, D, BF, "channel", True, seed=5)
    ref, tol = reference(small, 0.7, 1e-6, BF)
    big = {}
    for k, v in small.items():
        big[k] = v.cuda()
        if v.dim() == 2:
            big[k] = torch.zeros((n, D), dtype=BF, device="cuda")
            big[k][-last:] = v.cuda()
    out = {k: torch.empty((n, D), dtype=BF, device="cuda") for k in ("x_out", "u", "dx", "dy")}
    r1, r2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    par = dict(w_pre=big["w_pre"], w_post=big["w_post"], gate=big["gate"], res_scale=0.7, rstd_pre=r1, rstd_post=r2)
    dw = torch.empty(D, device="cuda")
    L.oomb_block_norm_fwd(big["x"], big["y"], out["x_out"], out["u"], eps=1e-6, **par)
    ws = torch.empty(L.oomb_block_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    L.oomb_block_norm_bwd(big["x"], big["y"], out["dx"], out["dy"], du=big["du"], dx_out=big["dx_out"], dw_pre=dw,
                          workspace=ws, **par)
    for k in out:
        compare({k: out[k][-last:]}, {k: ref[k]}, tol)
        assert not out[k][-last - 1].any()  # a row of zeros gives zeros
    compare({"dw_pre": dw}, {"dw_pre": ref["dw_pre"]}, {"dw_pre": tol["dw_pre"]})
