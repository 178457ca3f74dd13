"""Appends that continue the last page - token after token behind a prompt - against one append
of the same tokens, bit for bit; single-token attention over them; and what is refused."""
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


def make(dtype, Hq, Hkv, d, P, pages, **kw):
    pool = PagedKVPool(Hq, Hkv, d, P, pages, pages, dtype, "cuda",
                       page_order=torch.randperm(pages, generator=torch.Generator().manual_seed(pages)), **kw)
    pool.k_pool.fill_(math.nan)  # whatever stood there before
    pool.v_pool.fill_(math.nan)
    return pool


def contents(pool, n):
    pages = pool.table_host(-(-n // pool.P))
    return [t[pages].clone() for t in (pool.k_pool, pool.v_pool, pool.dk_pool, pool.dv_pool, pool.summary)]


@pytest.mark.parametrize("dtype,Hkv,d,P", [(BF, 4, 128, 128), (FP, 1, 64, 64), (BF, 2, 96, 48), (FP, 3, 20, 256),
                                           (BF, 1, 8, 2), (FP, 2, 128, 1)])
@pytest.mark.parametrize("cuts", [[1] * 9, [130, 1, 1, 1], [5, 600, 3], [127, 1, 1, 255, 1], [64, 192, 300]])
def test_the_same_bits_as_one_append(dtype, Hkv, d, P, cuts):
    N = sum(cuts)
    g = torch.Generator(device="cuda").manual_seed(N + d)
    k, v = (torch.randn(N, Hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    one, many = (make(dtype, Hkv, Hkv, d, P, -(-N // P)) for _ in range(2))
    L.oomb_kv_append(one.handle, k, v, 0)
    at = 0
    for n in cuts:
        L.oomb_kv_append(many.handle, k[at:at + n].contiguous(), v[at:at + n].contiguous(), at)
        at += n
        assert many.n_tokens == at
    assert L.oomb_check(one.handle) == 0 and L.oomb_check(many.handle) == 0
    assert one.table_host() == many.table_host()
    for a, b in zip(contents(one, N), contents(many, N)):
        assert not torch.isnan(a).any() and torch.equal(a, b)
    one.close(), many.close()


def test_gradients_in_front_stay():
    """The rows that are there keep their gradients, the new ones start from zero, whatever stood there."""
    pool = make(BF, 2, 2, 64, 32, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn(2, 60, 2, 64, generator=g, device="cuda").to(BF)
    L.oomb_kv_append(pool.handle, kv[0, :41].contiguous(), kv[1, :41].contiguous(), 0)
    pool.dk_pool.fill_(3.0)
    pool.dv_pool.fill_(4.0)
    L.oomb_kv_append(pool.handle, kv[0, 41:].contiguous(), kv[1, 41:].contiguous(), 41)
    for t, x in zip(pool.logical_grads(60), (3.0, 4.0)):
        assert (t[:41] == x).all() and (t[41:] == 0).all()
    pool.close()


@pytest.mark.parametrize("dtype,Hq,Hkv,d,P", [(BF, 14, 2, 128, 128), (FP, 2, 1, 64, 64)])
def test_token_after_token(dtype, Hq, Hkv, d, P):
    """A prompt that ends inside a page, then tokens one by one: selection, attention and append
    of each, against the float64 form."""
    prompt, new, top_k = 5 * P + 37, 2 * P - 30, 2
    N = prompt + new
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(N, Hkv, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(new, Hq, d, generator=g).to(dtype)
    slopes = 2.0 ** -(1.0 + torch.arange(Hq))
    kd, vd, qd, sd = k.cuda(), v.cuda(), q.cuda(), slopes.cuda()
    pool = make(dtype, Hq, Hkv, d, P, -(-N // P))
    h, scale = pool.handle, d ** -0.5
    L.oomb_kv_append(h, kd[:prompt].contiguous(), vd[:prompt].contiguous(), 0)
    ws, ws_sel = pool.workspace(L.OOMB_OP_SCORE_FWD, 1), pool.workspace(L.OOMB_OP_SELECT, 1)
    sel = torch.full((Hkv, top_k + 2), -1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(Hkv, dtype=torch.int32, device="cuda")
    for i in range(new):
        t = prompt + i
        L.oomb_kv_append(h, kd[t:t + 1], vd[t:t + 1], t)
        o, lse = torch.empty(1, Hq, d, dtype=dtype, device="cuda"), torch.empty(Hq, 1, device="cuda")
        L.oomb_page_select(h, qd[i:i + 1], t // P * P, top_k, 1, sel, cnt, ws_sel)
        L.oomb_score_attn_fwd(h, qd[i:i + 1], t, sel, cnt, scale, o, lse, ws, softcap=20.0, slopes=sd)
        if i % 29 and t % P not in (0, P - 1):
            continue
        assert L.oomb_check(h) == 0 and cnt.tolist() == [top_k + 2] * Hkv
        pages = sel.cpu().tolist()
        assert all(p[0] == 0 and p[-1] == t // P for p in pages)
        ref = score_attn(q[i:i + 1], k[:t + 1], v[:t + 1], pages, P, t, scale, 20.0, slopes,
                         tensor_cores=L.oomb_uses_tensor_cores(h))
        check("o", o, ref)
        check("lse", lse, ref)
    pool.close()


def test_refusals():
    pool = make(BF, 2, 2, 64, 32, 3)
    kv = torch.zeros(64, 2, 64, dtype=BF, device="cuda")
    ap = lambda n, at, p=pool: L.oomb_kv_append(p.handle, kv[:n], kv[:n], at)  # noqa: E731
    ap(40, 0)

    def refused(status, f, *a):
        with pytest.raises(L.OombError) as e:
            f(*a)
        assert e.value.status == status

    before = contents(pool, 40)
    refused(1, ap, 1, 39)    # not at the end
    refused(1, ap, 64, 40)   # more pages than the table has
    sel, cnt = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = pool.workspace(L.OOMB_OP_SELECT, 1)
    refused(3, L.oomb_page_select_append, pool.handle, kv[:1], kv[:1], kv[:1], 40, 1, 1, sel, cnt, ws)
    assert pool.n_tokens == 40
    for a, b in zip(before, contents(pool, 40)):
        assert torch.equal(a, b)
    L.oomb_page_free(pool.handle, 1, 1)
    refused(1, ap, 1, 40)    # the open page was freed
    pool.close()
    tight = PagedKVPool(2, 2, 64, 32, 2, 8, BF, "cuda")
    ap(40, 0, tight)
    refused(2, ap, 30, 40, tight)  # one page more than there are
    ap(24, 40, tight)              # the rest of the open one
    assert tight.n_tokens == 64 and L.oomb_check(tight.handle) == 0
    tight.close()
    off = PagedKVPool(2, 2, 64, 32, 3, 3, BF, "cuda", offload=True, stage_max_sel=3)
    ap(40, 0, off)
    refused(3, ap, 1, 40, off)  # pages in host memory are not continued
    L.oomb_check(off.handle)
    off.close()
