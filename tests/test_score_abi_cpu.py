"""Host-side refusals of the modified-score attention, the block norms and the multi-axis
rotation, through the C ABI on the CPU (placeholder pointers, never dereferenced), and the
Python calls' checks of their tensors."""
import ctypes as C

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300 import _lib, build

ARG, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 1, 3, 4, 8, 9
F = 1 << 24  # a placeholder address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return L.load()


@pytest.fixture(scope="module")
def pool(lib):
    d = _lib.PoolDesc()
    d.n_q_heads, d.n_kv_heads, d.head_dim, d.page_size = 28, 4, 128, 128
    d.num_phys_pages, d.max_logical_pages, d.dtype = 4, 8, _lib.OOMB_BF16
    for i, f in enumerate(["k_pool", "v_pool", "dk_pool", "dv_pool", "summary", "page_table", "error_word"]):
        setattr(d, f, (1 << 20) * (i + 1))
    h = L.oomb_pool_create(d)
    yield h
    L.oomb_pool_destroy(h)


def test_score_attn_refusals(lib, pool):
    mod = _lib.ScoreMod(30.0, None, None, None)
    fwd = lambda p=pool, q=F, q0=0, n=1, ms=4, m=mod, o=F: lib.oomb_score_attn_fwd(  # noqa: E731
        p, q, q0, n, F, F, ms, 0.1, C.byref(m), o, F, F, 1 << 40, None)
    assert fwd() == ARG  # nothing appended: the chunk's own K/V are not there
    assert fwd(p=None) == ARG and fwd(n=0) == ARG and fwd(q0=-1) == ARG and fwd(ms=0) == ARG and fwd(o=None) == ARG
    assert lib.oomb_score_attn_bwd(pool, F, F, F, F, 0, 1, F, F, 4, 0.1, None, F, F, 1 << 40, None) == ARG
    assert lib.oomb_score_attn_bwd(pool, F, F, None, F, 0, 1, F, F, 4, 0.1, None, F, F, 1 << 40, None) == ARG
    assert lib.oomb_workspace_size(pool, L.OOMB_OP_SCORE_BWD, 128) >= 28 * 128 * 4
    assert lib.oomb_workspace_size(pool, L.OOMB_OP_SCORE_FWD, 0) == 0
    assert lib.oomb_workspace_size(pool, 17, 128) == 0


@pytest.mark.parametrize("heads,dtype,d,P", [((28, 4), 0, 128, 128), ((2, 1), 1, 64, 64), ((300, 1), 0, 128, 128),
                                             ((40, 40), 0, 96, 32), ((4000, 2000), 0, 128, 128)])
def test_a_workspace_serves_every_smaller_call(lib, heads, dtype, d, P):
    """The sizes grow with n_q although fewer rows are cut into more parts."""
    de = _lib.PoolDesc()
    de.n_q_heads, de.n_kv_heads, de.head_dim, de.page_size = *heads, d, P
    de.num_phys_pages, de.max_logical_pages, de.dtype = 4, 8, dtype
    for i, f in enumerate(["k_pool", "v_pool", "dk_pool", "dv_pool", "summary", "page_table", "error_word"]):
        setattr(de, f, (1 << 20) * (i + 1))
    h = L.oomb_pool_create(de)
    for op in (L.OOMB_OP_SCORE_FWD, L.OOMB_OP_SCORE_BWD):
        sizes = [L.oomb_workspace_size(h, op, n) for n in [*range(1, 300), 513, 1000, 4097, 8192, 100000]]
        assert sizes == sorted(sizes)
    L.oomb_pool_destroy(h)


def test_doc_spans_refusals(lib):
    f = lib.oomb_doc_spans
    assert f(None, None, 1, 0, 4, F, F, None) == ARG
    assert f(F, None, 0, 0, 4, F, F, None) == ARG and f(F, None, 1, 0, 0, F, F, None) == ARG
    assert f(F, None, 1, -1, 4, F, F, None) == ARG and f(F, None, 2 ** 31 - 1, 0, 4, F, F, None) == ARG
    assert f(F + 4, None, 1, 0, 4, F, F, None) == ALIGN and f(F, F + 4, 1, 0, 4, F, F, None) == ALIGN


def test_block_norm_refusals(lib):
    def fwd(x=F, y=F, wp=F, g=F, rows=0, w=F, eps=1e-6, n=4, D=64, dt=0, xo=F, u=F, r1=None, r2=None):
        return lib.oomb_block_norm_fwd(x, y, wp, g, rows, w, 1.0, eps, n, D, dt, xo, u, r1, r2, None)

    assert fwd(x=None) == ARG and fwd(n=0) == ARG and fwd(D=0) == ARG and fwd(rows=2) == ARG
    assert fwd(y=None) == ARG  # a gate and a weight without the tensor they act on
    assert fwd(w=None) == ARG and fwd(u=None) == ARG  # u and its weight come together
    assert fwd(xo=None) == ARG and fwd(eps=-1.0) == ARG and fwd(eps=float("nan")) == ARG
    assert fwd(wp=None, r1=F) == ARG  # a statistic of a norm that is not there
    assert fwd(dt=5) == DTYPE and fwd(D=16385) == UNSUPPORTED
    assert fwd(x=F + 1) == ALIGN and fwd(w=F + 2) == ALIGN and fwd(g=F + 2) == ALIGN and fwd(xo=F + 1) == ALIGN

    def bwd(y=F, w=F, r1=F, r2=F, du=F, dxo=F, dx=F, dy=F, dwp=F, ws=F, nb=1 << 30, D=64):
        return lib.oomb_block_norm_bwd(F, y, F if y else None, F if y else None, 0, w, 1.0, 4, D, 0, r1, r2, du, dxo, dx,
                                       dy, dwp, None, None, 0, ws, nb, None)

    assert bwd(dx=None) == ARG and bwd(w=None) == ARG and bwd(du=None) == ARG
    assert bwd(r1=None) == ARG and bwd(r2=None) == ARG and bwd(y=None) == ARG
    assert bwd(w=None, du=None, dxo=None) == ARG  # no gradient arrives
    assert bwd(ws=None) == WORKSPACE and bwd(nb=64) == WORKSPACE and bwd(D=20000) == UNSUPPORTED
    assert bwd(dx=F + 1) == ALIGN and bwd(dwp=F + 2) == ALIGN and bwd(ws=F + 8) == ALIGN
    assert lib.oomb_block_norm_workspace(0, 64) == 0 and lib.oomb_block_norm_workspace(4, 64) >= 3 * 64 * 4


def test_rope_axes_refusals(lib):
    def f(x=F, o=F, ti=0, to=0, n=4, H=2, d=8, pos=F, A=2, axis=bytes([0, 1, 0, 1]), theta=1e4, lad=0, mode=1, bias=None):
        return lib.oomb_bias_rope_axes(x, ti, bias, o, to, n, H, d, pos, A, axis, theta, lad, mode, None)

    assert f(x=None) == ARG and f(n=0) == ARG and f(H=0) == ARG and f(d=7) == ARG and f(d=130) == ARG
    assert f(mode=3) == ARG and f(lad=2) == ARG and f(A=0) == ARG and f(A=9) == ARG and f(pos=None) == ARG
    assert f(axis=None) == ARG and f(axis=bytes([0, 1, 2, 0])) == ARG and f(theta=1.0) == ARG
    assert f(theta=float("nan")) == ARG and f(theta=float("inf")) == ARG
    assert f(ti=3) == DTYPE and f(to=3) == DTYPE and f(to=1) == ARG  # in place with two types
    assert f(x=F + 1, o=F) == ALIGN and f(pos=F + 4) == ALIGN and f(bias=F + 2) == ALIGN


def test_python_calls_refuse_host_tensors(lib, pool):
    """Tensors on the host never reach the library."""
    q = torch.zeros(1, 28, 128, dtype=torch.bfloat16)
    lse = torch.zeros(28, 1)
    sel, cnt = torch.zeros(4, 4, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        L.oomb_score_attn_fwd(pool, q, 0, sel, cnt, 0.1, q, lse)
    with pytest.raises(ValueError):
        L.oomb_score_attn_fwd(pool + 1, q, 0, sel, cnt, 0.1, q, lse)  # not a pool
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        L.oomb_block_norm_fwd(q[0], None, q[0].clone(), q[0].clone(), w_pre=torch.ones(128))
