"""Attention with modified scores over long selections: more pages than the tensor-core forward
looks up at once, than its ring of looked-up rows holds, and than a thread block has threads;
and workspaces, with what stands behind them, reused by calls of other sizes."""
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


class Setup:
    def __init__(self, dtype, Hq, Hkv, d, P, pages, n_q, drop, short=5):
        """The last page holds ``short`` tokens fewer than it could; each head leaves ``drop`` pages out."""
        g = torch.Generator(device="cuda").manual_seed(pages + n_q)
        self.N, self.n_q, self.P, self.Hq, self.Hkv = pages * P - short, n_q, P, Hq, Hkv
        self.q, self.do = (torch.randn(n_q, Hq, d, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.k, self.v = (torch.randn(self.N, Hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.pool = PagedKVPool(Hq, Hkv, d, P, pages, pages, dtype, "cuda",
                                page_order=torch.randperm(pages, generator=torch.Generator().manual_seed(1)))
        L.oomb_kv_append(self.pool.handle, self.k, self.v, 0)
        self.q0, self.scale = self.N - n_q, d ** -0.5
        own0 = self.q0 // P
        self.sel = []
        for h in range(Hkv):
            out = set(torch.randperm(own0, generator=torch.Generator().manual_seed(h))[:drop].tolist())
            self.sel.append([p for p in range(pages) if p not in out])
        self.dsel = torch.tensor(self.sel, dtype=torch.int32, device="cuda")
        self.cnt = torch.full((Hkv,), self.dsel.shape[1], dtype=torch.int32, device="cuda")

    def forward(self, ws=None, n=None, **mod):
        n = self.n_q if n is None else n
        q = self.q[-n:].contiguous()  # the last n rows
        o = torch.full_like(q, float("nan"))
        lse = torch.full((self.Hq, n), float("nan"), device="cuda")
        ws = self.pool.workspace(L.OOMB_OP_SCORE_FWD, n) if ws is None else ws
        L.oomb_score_attn_fwd(self.pool.handle, q, self.N - n, self.dsel, self.cnt, self.scale, o, lse, ws, **mod)
        return o, lse

    def backward(self, o, lse, ws=None, **mod):
        n = o.shape[0]
        self.pool.dk_pool.zero_(), self.pool.dv_pool.zero_()
        q, do, dq = self.q[-n:].contiguous(), self.do[-n:].contiguous(), torch.full_like(o, float("nan"))
        ws = self.pool.workspace(L.OOMB_OP_SCORE_BWD, n) if ws is None else ws
        L.oomb_score_attn_bwd(self.pool.handle, q, o, do, lse, self.N - n, self.dsel, self.cnt, self.scale, dq, ws, **mod)
        return dq, *self.pool.logical_grads(self.N)

    def close(self):
        self.pool.close()


def reference(s, cap, slopes, begin, end, train):
    with torch.device("cuda"):  # float64 sums of this size take the CPU minutes
        r = score_attn(s.q, s.k, s.v, s.sel, s.P, s.q0, s.scale, cap, slopes, begin, end, s.do if train else None,
                       tensor_cores=L.oomb_uses_tensor_cores(s.pool.handle))
    return {k: v.cpu() for k, v in r.items()}


SHAPES = {
    # more selected pages than threads; the keys cut over many thread blocks
    "rows_many_pages": dict(Hq=2, Hkv=1, pages=640, n_q=130, drop=20),
    "packed_many_pages": dict(Hq=8, Hkv=2, pages=640, n_q=3, drop=20),
    # one thread block walks every page of its tiles: rings longer than 64
    "rows_long_walk": dict(Hq=32, Hkv=4, pages=110, n_q=1100, drop=12),
    "packed_long_walk": dict(Hq=160, Hkv=160, pages=150, n_q=2, drop=10),
}


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("mask", ["causal", "cut"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_long_selections(shape, mask, cap, bias):
    s = Setup(BF, d=128, P=128, **SHAPES[shape])
    slopes = 2.0 ** (-12.0 * (torch.arange(s.Hq, device="cuda") % 8 + 1) / 8) if bias else None
    begin = end = None
    if mask == "cut":  # from anywhere in the first third up to the row, or past it
        g = torch.Generator(device="cuda").manual_seed(2)
        begin = torch.randint(0, s.N // 3, (s.n_q,), generator=g, device="cuda")
        end = torch.arange(s.q0, s.N, device="cuda") + 1 + torch.randint(0, 300, (s.n_q,), generator=g, device="cuda")
    mod = dict(softcap=cap, slopes=slopes, key_begin=begin, key_end=end)
    train = shape != "packed_long_walk"
    o, lse = s.forward(**mod)
    ref = reference(s, cap, slopes, begin, end, train)
    assert L.oomb_check(s.pool.handle) == 0
    check("o", o, ref)
    check("lse", lse, ref)
    if train:
        got = s.backward(o, lse, **mod)
        assert L.oomb_check(s.pool.handle) == 0
        for name, x in zip(("dq", "dk", "dv"), got):
            check(name, x, ref)
    s.close()


@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,pages", [(BF, 14, 2, 128, 128, 20), (BF, 8, 8, 128, 128, 40),
                                                    (FP, 2, 1, 64, 64, 30), (BF, 6, 2, 96, 32, 30), (FP, 6, 2, 128, 16, 30)])
def test_workspaces_of_larger_calls(dtype, Hq, Hkv, d, P, pages):
    """Every smaller call gives the bits that it gives with a workspace of its own, and writes
    nothing behind the size that was handed out."""
    most = min(700, pages * P - 10)
    s = Setup(dtype, Hq, Hkv, d, P, pages, most, drop=0)
    mod = dict(softcap=15.0, slopes=2.0 ** -(1.0 + torch.arange(Hq, device="cuda") % 8))
    behind = 1 << 16
    spaces = []
    for op in (L.OOMB_OP_SCORE_FWD, L.OOMB_OP_SCORE_BWD):
        size = L.oomb_workspace_size(s.pool.handle, op, most)
        spaces.append(torch.full((size + behind,), 0xA5, dtype=torch.uint8, device="cuda"))
    for n in (most, 1, 2, 9, 18, 63, 65, 100, 129, 256, 300, most):
        o, lse = s.forward(n=n, **mod)
        dq, dk, dv = (t.clone() for t in s.backward(o, lse, **mod))
        fwd, bwd = (w[:-behind] for w in spaces)
        o2, lse2 = s.forward(ws=fwd, n=n, **mod)
        dq2, dk2, dv2 = s.backward(o2, lse2, ws=bwd, **mod)
        assert L.oomb_check(s.pool.handle) == 0
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and not torch.isnan(o).any()
        assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
        if L.oomb_uses_tensor_cores(s.pool.handle):  # dq is summed in no fixed order there
            assert (dq.float() - dq2.float()).norm() <= 2.0 ** -8 * dq.float().norm()
        else:
            assert torch.equal(dq, dq2)
        assert all((w[-behind:] == 0xA5).all() for w in spaces)
    s.close()
