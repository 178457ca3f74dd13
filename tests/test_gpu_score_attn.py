"""Chunk attention with capped scores, distance bias and per-row key ranges on the GPU
against its float64 form: forward, backward, both kernel families, the ranges' edges."""
import math

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300.pool import PagedKVPool

from score_ref import check, score_attn

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ranges(kind, n_q, q_start, total, seed=0):
    """Key ranges of a test: None, or (key_begin, key_end), either of them None."""
    pos = torch.arange(q_start, q_start + n_q)
    if kind == "causal":
        return None, None
    if kind == "window":  # the last 50 tokens only
        return (pos - 49).clamp(min=0), None
    if kind == "docs":
        return pos // 90 * 90, pos + 1
    if kind == "prefix":  # keys behind the row's own position, up to the end of the cache
        return None, torch.maximum(pos + 1, torch.full_like(pos, min(total, q_start + n_q + 70)))
    if kind == "empty":  # every third row sees nothing, one way or another
        b, e = pos // 100 * 100, pos + 1
        e = torch.where(pos % 3 == 0, b, e)
        return b, torch.where(pos % 9 == 0, b - 5, e)
    if kind == "none":
        return pos * 0 + total, pos * 0
    if kind == "beyond":  # cut to the tokens there are
        return pos * 0 - 1000, pos * 0 + (1 << 40)
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, total, (n_q,), generator=g)
    return b, b + torch.randint(0, 200, (n_q,), generator=g)


def selection(kind, Hkv, n_pages, own0, seed):
    g = torch.Generator().manual_seed(seed)
    rows = []
    for h in range(Hkv):
        if kind == "all":
            rows.append(list(range(n_pages)))
        elif kind == "own":
            rows.append(list(range(own0, n_pages)))
        else:  # the first page, some history, not the same for every head, and the rest
            keep = [p for p in range(1, own0) if torch.rand(1, generator=g).item() < 0.5]
            rows.append(([0] if own0 > 0 else []) + keep + list(range(own0, n_pages)))
    return rows


class Case:
    def __init__(self, dtype, Hq, Hkv, d, P, total, n_q, q_start=None, sel="some", cap=0.0, bias=False, mask="causal",
                 seed=0, spread=1.0, offload=False):
        g = torch.Generator().manual_seed(1000 + seed)
        self.q_start = total - n_q if q_start is None else q_start
        self.dtype, self.P, self.total, self.n_q = dtype, P, total, n_q
        self.q = (torch.randn(n_q, Hq, d, generator=g) * spread).to(dtype)
        self.k = torch.randn(total, Hkv, d, generator=g).to(dtype)
        self.v = torch.randn(total, Hkv, d, generator=g).to(dtype)
        self.do = torch.randn(n_q, Hq, d, generator=g).to(dtype)
        self.scale = 1.0 / math.sqrt(d)
        self.cap = cap
        self.slopes = (2.0 ** (-4.0 * (torch.arange(Hq, dtype=FP) + 1) / Hq)) if bias else None
        self.begin, self.end = ranges(mask, n_q, self.q_start, total, seed)
        n_pages = -(-total // P)
        view = n_pages if self.end is not None else -(-(self.q_start + n_q) // P)
        self.sel = selection(sel, Hkv, view, self.q_start // P, seed)
        self.order = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.pool = PagedKVPool(Hq, Hkv, d, P, n_pages, n_pages, dtype, "cuda", page_order=self.order)
        self.dev = self.pool.device
        L.oomb_kv_append(self.pool.handle, self.k.cuda(), self.v.cuda(), 0)
        width = max(1, max(len(r) for r in self.sel)) + 2  # entries behind the count are never read
        self.dsel = torch.full((Hkv, width), -7, dtype=torch.int32)
        for h, r in enumerate(self.sel):
            self.dsel[h, :len(r)] = torch.tensor(r, dtype=torch.int32)
        self.dsel = self.dsel.cuda()
        self.cnt = torch.tensor([len(r) for r in self.sel], dtype=torch.int32).cuda()
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.mod = dict(softcap=cap, slopes=up(self.slopes), key_begin=up(self.begin), key_end=up(self.end))
        self.dq_in = self.q.cuda()

    def forward(self, stream=None):
        o = torch.full_like(self.dq_in, float("nan"))
        lse = torch.full((self.q.shape[1], self.n_q), float("nan"), device="cuda")
        ws = self.pool.workspace(L.OOMB_OP_SCORE_FWD, self.n_q)
        L.oomb_score_attn_fwd(self.pool.handle, self.dq_in, self.q_start, self.dsel, self.cnt, self.scale, o, lse, ws,
                              stream=stream, **self.mod)
        return o, lse

    def backward(self, o, lse):
        dq = torch.full_like(self.dq_in, float("nan"))
        ws = self.pool.workspace(L.OOMB_OP_SCORE_BWD, self.n_q)
        L.oomb_score_attn_bwd(self.pool.handle, self.dq_in, o, self.do.cuda(), lse, self.q_start, self.dsel, self.cnt,
                              self.scale, dq, ws, **self.mod)
        return dq

    def reference(self, train=True):
        tc = L.oomb_uses_tensor_cores(self.pool.handle)
        return score_attn(self.q, self.k, self.v, self.sel, self.P, self.q_start, self.scale, self.cap, self.slopes,
                          self.begin, self.end, self.do if train else None, tensor_cores=tc)

    def run(self, train=True):
        ref = self.reference(train)
        o, lse = self.forward()
        if train:
            dq = self.backward(o, lse)
        assert L.oomb_check(self.pool.handle) == 0
        check("o", o, ref)
        check("lse", lse, ref)
        if train:
            dk, dv = self.pool.logical_grads(self.total)
            check("dq", dq, ref)
            check("dv", dv, ref)
            check("dk", dk, ref)
        self.pool.close()


TC = dict(dtype=BF, d=128, P=128)  # the tensor-core shape

SHAPES = {
    "tc_g2_ragged": dict(TC, Hq=4, Hkv=2, total=900, n_q=300),
    "tc_g7_unaligned": dict(TC, Hq=7, Hkv=1, total=700, n_q=131, q_start=333),
    "tc_g1": dict(TC, Hq=2, Hkv=2, total=520, n_q=256),
    "tc_one_token": dict(TC, Hq=14, Hkv=2, total=1500, n_q=1),
    "tc_few_tokens": dict(TC, Hq=14, Hkv=2, total=1301, n_q=18),
    "tc_few_tokens_inside": dict(TC, Hq=14, Hkv=2, total=1301, n_q=19, q_start=640),
    "tc_first_token": dict(TC, Hq=4, Hkv=2, total=1, n_q=1),
    "tc_wide_group": dict(TC, Hq=40, Hkv=1, total=300, n_q=5),
    "fp32_64": dict(dtype=FP, d=64, P=64, Hq=2, Hkv=1, total=777, n_q=200),
    "fp32_small_pages": dict(dtype=FP, d=128, P=16, Hq=6, Hkv=2, total=400, n_q=70, q_start=301),
    "fp32_page_1": dict(dtype=FP, d=20, P=1, Hq=3, Hkv=3, total=130, n_q=65),
    "fp32_large_pages": dict(dtype=FP, d=32, P=256, Hq=4, Hkv=1, total=1000, n_q=3),
    "bf16_odd_page": dict(dtype=BF, d=96, P=48, Hq=4, Hkv=2, total=431, n_q=129),
    "bf16_d8": dict(dtype=BF, d=8, P=32, Hq=2, Hkv=2, total=97, n_q=97),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True), (30.0, True)])
def test_scores_match(shape, cap, bias):
    Case(cap=cap, bias=bias, **SHAPES[shape]).run()


@pytest.mark.parametrize("mask", ["window", "docs", "prefix", "empty", "none", "beyond", "random"])
@pytest.mark.parametrize("shape", ["tc_g2_ragged", "tc_g7_unaligned", "tc_few_tokens_inside", "fp32_64",
                                   "fp32_small_pages", "bf16_odd_page"])
def test_ranges_match(shape, mask):
    Case(cap=20.0, bias=True, mask=mask, sel="all", seed=3, **SHAPES[shape]).run()


@pytest.mark.parametrize("sel", ["all", "own", "some"])
@pytest.mark.parametrize("mask", ["docs", "random"])
def test_ranges_meet_selections(sel, mask):
    """Rows whose range holds no selected page, heads with different pages."""
    Case(mask=mask, sel=sel, seed=5, total=1400, n_q=390, q_start=700, Hq=4, Hkv=2, **TC).run()


@pytest.mark.parametrize("cap", [255.0, 257.0, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("shape", ["tc_g2_ragged", "tc_few_tokens", "fp32_64"])
def test_cap_far_above_the_scores(shape, cap):
    """A cap that hardly bends the scores: held to bounds in which the cap itself has no part
    (an error of 2^-23 of the cap would not do): the uncapped form, which differs by
    |s|^3 / (3 cap^2), or above 1e3 not at all."""
    c = Case(cap=cap, bias=True, mask="docs", sel="all", **SHAPES[shape])
    c.cap, exact_cap = 0.0, c.cap
    if cap < 1e3:
        c.cap = exact_cap
    c.run()


@pytest.mark.parametrize("shape", ["tc_g2_ragged", "tc_few_tokens", "fp32_64"])
def test_tiny_cap(shape):
    """Scores that are all but the sign of the dot product; zero queries stay zero."""
    c = Case(cap=1e-3, **SHAPES[shape])
    c.q[::2] = 0
    c.dq_in = c.q.cuda()
    o, lse = c.forward()
    dq = c.backward(o, lse)
    assert L.oomb_check(c.pool.handle) == 0
    ref = c.reference(False)
    check("o", o, ref)
    check("lse", lse, ref)
    assert torch.isfinite(dq.float()).all()
    c.pool.close()


@pytest.mark.parametrize("mask", ["docs", "random", "empty"])
def test_more_tiles_than_fit_the_gpu_at_once(mask):
    """Ranges and enough query tiles for several waves of thread blocks."""
    Case(mask=mask, sel="all", bias=True, cap=15.0, total=1400, n_q=1100, Hq=32, Hkv=4, **TC).run()


@pytest.mark.parametrize("spread", [0.01, 30.0])
@pytest.mark.parametrize("shape", ["tc_g2_ragged", "fp32_64"])
def test_cap_small_and_saturated(shape, spread):
    """Arguments of the tanh far below and far above 1."""
    Case(cap=4.0, spread=spread, **SHAPES[shape]).run()


def spans_of(cuts, pre, q_start, n_q):
    out = []
    for t in range(q_start, q_start + n_q):
        doc = [c for c in range(len(cuts) - 1) if cuts[c] <= t < cuts[c + 1]]
        if not doc:
            out.append((t, t))
            continue
        c = doc[0]
        e = t + 1 if pre is None else max(t + 1, min(cuts[c] + pre[c], cuts[c + 1]))
        out.append((cuts[c], e))
    return torch.tensor(out, dtype=torch.int64)


@pytest.mark.parametrize("cuts,pre", [
    ([0, 5, 5, 9, 40], None), ([0, 5, 5, 9, 40], [3, 0, 100, 10]), ([10, 30], [-4]), ([0, 1000], [1 << 62]),
    ([7, 7], None), ([3, 4, 5, 6], [1, 1, 1])])
def test_doc_spans(cuts, pre):
    """Empty documents, rows before the first and behind the last one, prefixes past their document."""
    for q_start, n_q in ((0, 50), (4, 1), (33, 300)):
        b = torch.full((n_q,), -1, dtype=torch.int64, device="cuda")
        e = torch.full((n_q,), -1, dtype=torch.int64, device="cuda")
        up = lambda v: None if v is None else torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731
        L.oomb_doc_spans(up(cuts), q_start, b, e, prefix_len=up(pre))
        assert torch.equal(torch.stack([b, e], 1).cpu(), spans_of(cuts, pre, q_start, n_q))


@pytest.mark.parametrize("shape", ["tc_g2_ragged", "fp32_64"])
def test_without_a_modification_it_is_chunk_attention(shape):
    """No cap, bias or ranges: the plain causal attention of a chunk that starts on a page."""
    kw = dict(SHAPES[shape], total=512 + 300, n_q=300)
    c = Case(**kw)
    o, lse = c.forward()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    L.oomb_chunk_attn_fwd(c.pool.handle, c.dq_in, c.q_start, c.dsel, c.cnt, c.scale, o2, lse2)
    L.oomb_check(c.pool.handle)
    ref = c.reference(False)
    ref["o_tol"] = 2 * ref["o_tol"]
    check("o", o2, {**ref, "o": o.double().cpu()})
    check("lse", lse2, {**ref, "lse": lse.double().cpu(), "lse_tol": 2 * ref["lse_tol"]})
    c.pool.close()


def test_gradients_of_the_reference_against_differences():
    """The float64 form the kernels are held to, by central differences of its forward."""
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(5, 2, 4, generator=g).double(), torch.randn(7, 1, 4, generator=g).double(),
                   torch.randn(7, 1, 4, generator=g).double(), torch.randn(5, 2, 4, generator=g).double())
    b, e = torch.tensor([0, 1, 2, 0, 3]), torch.tensor([3, 4, 7, 0, 6])
    arg = dict(sel=[[0, 1, 3]], P=2, q_start=2, scale=0.5, cap=1.5, slopes=torch.tensor([0.3, 0.1]), key_begin=b,
               key_end=e)
    ref = score_attn(q, k, v, do=do, **arg)
    x = {"q": q, "k": k, "v": v}
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        for i in range(0, x[name].numel(), 3):
            val = []
            for h in (1e-5, -1e-5):
                y = {n: t.clone() for n, t in x.items()}
                y[name].view(-1)[i] += h
                val.append((score_attn(y["q"], y["k"], y["v"], **arg)["o"] * do).sum().item())
            num = (val[0] - val[1]) / 2e-5
            assert abs(num - ref[grad].view(-1)[i].item()) < 1e-7 * (1 + abs(num)), (name, i)


def test_gradients_add_to_what_the_pool_holds_and_repeat():
    """Two backwards add twice; dK and dV are the same bits on every run."""
    for shape in ("tc_g2_ragged", "bf16_odd_page"):
        c = Case(cap=10.0, bias=True, mask="docs", sel="all", **SHAPES[shape])
        o, lse = c.forward()
        c.backward(o, lse)
        one = [t.clone() for t in c.pool.logical_grads(c.total)]
        c.backward(o, lse)
        two = [t.clone() for t in c.pool.logical_grads(c.total)]
        assert L.oomb_check(c.pool.handle) == 0
        for a, b in zip(one, two):
            assert torch.equal(b, a + a)
        c.pool.close()


def test_bad_selections_are_flagged_and_left_out():
    """An unmapped page and entries out of order: flagged, nothing else is touched."""
    c = Case(sel="all", total=640, n_q=128, Hq=4, Hkv=2, **TC)
    L.oomb_page_free(c.pool.handle, 1, 1)
    o, lse = c.forward()
    with pytest.raises(L.OombError):
        L.oomb_check(c.pool.handle)
    c.sel = [[p for p in r if p != 1] for r in c.sel]
    ref = c.reference(False)
    check("o", o, ref)
    check("lse", lse, ref)
    for row in ([0, 3, 2, 4], [0, 2, 2, 4], [-1, 0, 2, 4], [0, 2, 4, 5], [0, 2, 4, 1 << 30]):
        c.dsel[0, :4] = torch.tensor(row, dtype=torch.int32)
        c.cnt.fill_(4)
        o, lse = c.forward()
        with pytest.raises(L.OombError):
            L.oomb_check(c.pool.handle)
        c.backward(o, lse)
        with pytest.raises(L.OombError):
            L.oomb_check(c.pool.handle)
    c.cnt.fill_(c.dsel.shape[1] + 1)  # a count past the row
    c.forward()
    with pytest.raises(L.OombError):
        L.oomb_check(c.pool.handle)
    c.cnt.fill_(0)  # no pages at all
    o, lse = c.forward()
    assert L.oomb_check(c.pool.handle) == 0
    assert not o.any() and torch.isinf(lse).all() and not c.backward(o, lse).any()
    c.pool.close()


@pytest.mark.parametrize("n_q", [1, 200])
def test_what_a_page_left_out_holds_does_not_matter(n_q):
    """An unmapped page in the selection, and NaN in every block of the pools that no page uses."""
    c = Case(sel="all", total=640, n_q=n_q, Hq=4, Hkv=2, **TC)
    table = L.oomb_page_table_host(c.pool.handle, 5)
    gone = min(range(4), key=lambda p: int(table[p]))
    L.oomb_page_free(c.pool.handle, gone, 1)
    for pool in (c.pool.k_pool, c.pool.v_pool):
        pool[[i for i in range(pool.shape[0]) if i not in [int(table[p]) for p in range(5) if p != gone]]] = math.nan
    o, lse = c.forward()
    with pytest.raises(L.OombError):
        L.oomb_check(c.pool.handle)
    c.sel = [[p for p in r if p != gone] for r in c.sel]
    ref = c.reference(False)
    check("o", o, ref)
    check("lse", lse, ref)
    c.pool.close()


def test_refusals():
    c = Case(total=300, n_q=40, Hq=4, Hkv=2, **TC)
    h, q, o = c.pool.handle, c.dq_in, torch.empty_like(c.dq_in)
    lse = torch.empty(4, 40, device="cuda")
    ws = c.pool.workspace(L.OOMB_OP_SCORE_FWD, 40)
    call = lambda **kw: L.oomb_score_attn_fwd(h, kw.pop("q", q), kw.pop("q0", c.q_start), kw.pop("sel", c.dsel),  # noqa: E731
                                              c.cnt, 0.1, o, kw.pop("lse", lse), kw.pop("ws", ws), **kw)
    call()
    for kw in (dict(q=q[:, :, ::2]), dict(q=q[:, :3]), dict(q=q.cpu()), dict(lse=lse[:, :39]), dict(sel=c.dsel[:1]),
               dict(key_begin=torch.zeros(39, dtype=torch.int64, device="cuda")),
               dict(slopes=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=q.float()), dict(sel=c.dsel.long()), dict(key_end=torch.zeros(40, device="cuda"))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e31),
               dict(softcap=1e-35), dict(q0=261), dict(q0=-1)):
        with pytest.raises(L.OombError) as e:
            call(**kw)
        assert e.value.status == 1
    if ws.numel() > 16:
        with pytest.raises(L.OombError) as e:
            call(ws=ws[:16])
        assert e.value.status == 9
    with pytest.raises(L.OombError) as e:
        L.oomb_score_attn_bwd(h, q, o, o, lse, c.q_start, c.dsel, c.cnt, 0.1, torch.empty_like(q), ws[:16])
    assert e.value.status == 9
    L.oomb_check(h)
    c.pool.close()


def test_other_stream_and_graph_replay():
    """Forward and backward on a side stream, and captured once and replayed on other inputs;
    two graphs with a workspace each, replayed at the same time."""
    kw = dict(TC, total=800, n_q=290, Hq=4, Hkv=2, cap=12.0, bias=True, mask="docs", sel="all")
    eager = []
    for seed in (1, 2):
        c = Case(seed=seed, **kw)
        o, lse = c.forward()
        dq = c.backward(o, lse)
        eager.append((o, lse, dq, *[t.clone() for t in c.pool.logical_grads(c.total)]))
        c.pool.close()
    side = torch.cuda.Stream()
    graphs, alive = [], []
    for seed in (1, 2):
        c = Case(seed=seed, **kw)
        do, out = c.do.cuda(), {}
        ws = [c.pool.workspace(op, c.n_q) for op in (L.OOMB_OP_SCORE_FWD, L.OOMB_OP_SCORE_BWD)]
        out["o"], out["dq"] = torch.empty_like(c.dq_in), torch.empty_like(c.dq_in)
        out["lse"] = torch.empty(4, c.n_q, device="cuda")

        def step(c=c, do=do, out=out, ws=ws):
            c.pool.dk_pool.zero_()
            c.pool.dv_pool.zero_()
            a = (c.dsel, c.cnt, c.scale)
            L.oomb_score_attn_fwd(c.pool.handle, c.dq_in, c.q_start, *a, out["o"], out["lse"], ws[0], **c.mod)
            L.oomb_score_attn_bwd(c.pool.handle, c.dq_in, out["o"], do, out["lse"], c.q_start, *a, out["dq"], ws[1],
                                  **c.mod)

        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # on the side stream, eagerly
        side.synchronize()
        assert torch.equal(out["o"], eager[seed - 1][0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, c, out))
        alive.append(step)  # holds the inputs and the workspaces that the graph uses
    for _ in range(3):
        for g, c, out in graphs:
            out["o"].zero_(), out["dq"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        graphs[1][0].replay()
        torch.cuda.synchronize()
        for (g, c, out), ref in zip(graphs, eager):
            assert torch.equal(out["o"], ref[0]) and torch.equal(out["lse"], ref[1])
            dk, dv = c.pool.logical_grads(c.total)
            assert torch.equal(dk, ref[3]) and torch.equal(dv, ref[4])
            # dq is summed in no fixed order: a few fp32 additions apart, then one rounding
            assert (out["dq"].float() - ref[2].float()).norm() <= 2.0 ** -8 * ref[2].float().norm()
    # the same graph on other queries
    g, c, out = graphs[0]
    c.q = torch.flip(c.q, (0,)).contiguous()
    c.dq_in.copy_(c.q)
    g.replay()
    assert L.oomb_check(c.pool.handle) == 0
    ref = c.reference(False)
    check("o", out["o"], ref)
    for g, c, out in graphs:
        c.pool.close()


def test_offload_pool_matches_resident():
    """K/V and gradients in host memory: the staged blocks give the resident pool's bits."""
    kw = dict(TC, total=900, n_q=260, q_start=640, Hq=4, Hkv=2, cap=9.0, bias=True, mask="docs")
    c = Case(**kw)
    o, lse = c.forward()
    c.backward(o, lse)
    dk, dv = (t.clone() for t in c.pool.logical_grads(c.total))
    n_pages = -(-c.total // c.P)
    width = c.dsel.shape[1]
    off = PagedKVPool(4, 2, 128, 128, n_pages, n_pages, BF, "cuda", page_order=c.order, offload=True,
                      stage_max_sel=width, offload_grads=True)
    h = off.handle
    L.oomb_kv_append(h, c.k.cuda(), c.v.cuda(), 0)
    L.oomb_prefetch(h, c.dsel, c.cnt, 1)
    L.oomb_grad_prefetch(h, c.dsel, c.cnt, None, None, 1)
    L.oomb_pool_set_stage(h, 1)
    o2, lse2, dq2 = torch.empty_like(o), torch.empty_like(lse), torch.empty_like(o)
    ws = off.workspace(L.OOMB_OP_SCORE_FWD, c.n_q)
    a = (c.dsel, c.cnt, c.scale)
    L.oomb_score_attn_fwd(h, c.dq_in, c.q_start, *a, o2, lse2, ws, **c.mod)
    L.oomb_score_attn_bwd(h, c.dq_in, o2, c.do.cuda(), lse2, c.q_start, *a, dq2,
                          off.workspace(L.OOMB_OP_SCORE_BWD, c.n_q), **c.mod)
    L.oomb_grad_writeback(h, c.dsel, c.cnt, 1)
    assert L.oomb_check(h) == 0 and L.oomb_check(c.pool.handle) == 0
    dk2, dv2 = off.logical_grads(c.total)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(dk.cpu(), dk2.cpu()) and torch.equal(dv.cpu(), dv2.cpu())
    off.close()
    c.pool.close()


def test_one_workspace_for_calls_of_every_size():
    """A workspace of the largest call serves the smaller ones, which cut their keys finer."""
    big = Case(sel="all", total=2000, n_q=700, Hq=14, Hkv=2, cap=10.0, **TC)
    ws = big.pool.workspace(L.OOMB_OP_SCORE_FWD, 700)
    for n in (1, 9, 18, 100, 256, 300, 700):
        q = big.dq_in[:n].contiguous()
        o = torch.full_like(q, float("nan"))
        lse = torch.full((14, n), float("nan"), device="cuda")
        guard = ws.clone().fill_(7)
        L.oomb_score_attn_fwd(big.pool.handle, q, big.q_start, big.dsel, big.cnt, big.scale, o, lse, guard, softcap=10.0)
        ref = score_attn(big.q[:n], big.k, big.v, [[p for p in r if p * 128 < big.q_start + n] for r in big.sel], 128,
                         big.q_start, big.scale, 10.0)
        if n < 700:  # pages of the full chunk are past this call's view: flagged
            with pytest.raises(L.OombError):
                L.oomb_check(big.pool.handle)
        check("o", o, ref)
        check("lse", lse, ref)
    big.pool.close()


def test_rows_behind_the_last_and_buffers_around_are_left_alone():
    """Nothing is written outside O, LSE, dq and the touched pages."""
    c = Case(sel="own", total=700, n_q=77, q_start=560, Hq=4, Hkv=2, cap=5.0, **TC)
    pad = 4
    box = torch.full((c.n_q + 2 * pad, 4, 128), 3.0, dtype=BF, device="cuda")
    lbox = torch.full((4 * c.n_q + 64,), 3.0, device="cuda")
    o, lse = box[pad:pad + c.n_q], lbox[32:32 + 4 * c.n_q].view(4, c.n_q)
    L.oomb_score_attn_fwd(c.pool.handle, c.dq_in, c.q_start, c.dsel, c.cnt, c.scale, o, lse,
                          c.pool.workspace(L.OOMB_OP_SCORE_FWD, c.n_q), **c.mod)
    qbox = torch.full_like(box, 3.0)
    L.oomb_score_attn_bwd(c.pool.handle, c.dq_in, o, c.do.cuda(), lse, c.q_start, c.dsel, c.cnt, c.scale,
                          qbox[pad:pad + c.n_q], c.pool.workspace(L.OOMB_OP_SCORE_BWD, c.n_q), **c.mod)
    assert L.oomb_check(c.pool.handle) == 0
    for b in (box, qbox):
        assert (b[:pad] == 3).all() and (b[-pad:] == 3).all()
    assert (lbox[:32] == 3).all() and (lbox[-32:] == 3).all()
    dk, dv = c.pool.logical_grads(c.total)
    first = min(c.sel[0]) * 128
    assert not dk[:first].any() and not dv[:first].any() and not dk[637:].any() and not dv[637:].any()
    c.pool.close()


@pytest.mark.parametrize("dtype,n_q", [(BF, 5), (BF, 300), (FP, 130)])
def test_offsets_past_32_bits(dtype, n_q):
    """Pages whose elements stand more than 2^31 from the pools' start."""
    H, pages, chunk = 8, 16500, 125
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn(chunk * 128, H, 128, generator=g).to(dtype) for _ in range(2))
    q, do = (torch.randn(n_q, H, 128, generator=g).to(dtype) for _ in range(2))
    pool = PagedKVPool(H, H, 128, 128, pages, pages, dtype)
    kd, vd = k.cuda(), v.cuda()
    for first in range(0, pages, chunk):
        L.oomb_kv_append(pool.handle, kd, vd, first * 128)
    sel = [0, 7, 16390, 16444] + list(range(pages - 3, pages))
    q0 = pages * 128 - n_q
    dsel = torch.tensor([sel] * H, dtype=torch.int32).cuda()
    cnt = torch.full((H,), len(sel), dtype=torch.int32).cuda()
    qd, o, dq = q.cuda(), torch.empty_like(q, device="cuda"), torch.empty_like(q, device="cuda")
    lse = torch.empty(H, n_q, device="cuda")
    a = (q0, dsel, cnt, 0.09)
    L.oomb_score_attn_fwd(pool.handle, qd, *a, o, lse, pool.workspace(L.OOMB_OP_SCORE_FWD, n_q), softcap=12.0)
    L.oomb_score_attn_bwd(pool.handle, qd, o, do.cuda(), lse, *a, dq, pool.workspace(L.OOMB_OP_SCORE_BWD, n_q),
                          softcap=12.0)
    assert L.oomb_check(pool.handle) == 0
    # the same keys one after another: only the last pages are behind or beside the queries
    kc, vc = (torch.cat([t[p % chunk * 128:p % chunk * 128 + 128] for p in sel]) for t in (k, v))
    ref = score_attn(q, kc, vc, [list(range(len(sel)))] * H, 128, kc.shape[0] - n_q, 0.09, 12.0, do=do,
                     tensor_cores=dtype == BF)
    table = L.oomb_page_table_host(pool.handle, pages)
    dk, dv = (torch.cat([t[table[p]].permute(1, 0, 2) for p in sel]) for t in (pool.dk_pool, pool.dv_pool))
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got, ref)
    pool.close()
