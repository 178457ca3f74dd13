"""Host-side refusals of the embeddings, layer norm and the loss over a vocabulary, through the C ABI
on the CPU (placeholder pointers, never dereferenced), and the Python calls' checks of their tensors."""
import ctypes as C

import pytest
import torch

import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300 import build

ARG, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 1, 3, 4, 8, 9
F = 1 << 24  # a placeholder address
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    build.build()
    return L.load()


def refused(call, status, **cases):
    for name, values in cases.items():
        for v in values if isinstance(values, (list, tuple)) else [values]:
            assert call(**{name: v}) == status, (name, v)


def test_embed_refusals(lib):
    def fwd(tokens=F, n=4, table=F, V=10, D=8, dtype=0, scale=1.0, out=F, word=F):
        return lib.oomb_embed_fwd(tokens, n, table, V, D, dtype, scale, out, word, None)

    def bwd(tokens=F, n=4, d_out=F, V=10, D=8, dtype=0, scale=1.0, d_table=F, ws=F, size=BIG, word=F):
        return lib.oomb_embed_bwd(tokens, n, d_out, V, D, dtype, scale, d_table, 1, ws, size, word, None)

    inf, nan = float("inf"), float("nan")
    for call in (fwd, bwd):
        refused(call, ARG, tokens=None, n=[0, -1], V=[0, -5, 2 ** 31 - 1], D=[0, -1], scale=[inf, nan], word=None)
        refused(call, DTYPE, dtype=[2, -1])
        refused(call, ALIGN, tokens=F + 4, word=F + 2)
        refused(call, UNSUPPORTED, D=(1 << 24) + 1)
    refused(fwd, ARG, table=None, out=None)
    refused(fwd, ALIGN, table=F + 1, out=F + 1)
    refused(bwd, ARG, d_out=None, d_table=None)
    refused(bwd, ALIGN, d_out=F + 1, d_table=F + 2, ws=F + 8)
    refused(bwd, WORKSPACE, ws=None, size=[0, lib.oomb_embed_workspace(4, 8) - 1])
    assert lib.oomb_embed_workspace(0, 8) == 0 and lib.oomb_embed_workspace(4, 0) == 0


def test_layer_norm_refusals(lib):
    def fwd(x=F, w=F, b=F, eps=1e-5, n=4, D=8, dtype=0, out=F, mean=F, rstd=F):
        return lib.oomb_layer_norm_fwd(x, w, b, eps, n, D, dtype, out, mean, rstd, None)

    def bwd(x=F, w=F, mean=F, rstd=F, dy=F, dx_out=F, n=4, D=8, dtype=0, dx=F, dw=F, db=F, ws=F, size=BIG):
        return lib.oomb_layer_norm_bwd(x, w, mean, rstd, dy, dx_out, n, D, dtype, dx, dw, db, 0, ws, size, None)

    for call in (fwd, bwd):
        refused(call, ARG, x=None, n=[0, -2], D=[0, -1])
        refused(call, DTYPE, dtype=3)
        refused(call, UNSUPPORTED, D=16385)
        refused(call, ALIGN, x=F + 1, w=F + 2, mean=F + 1, rstd=F + 2)
    refused(fwd, ARG, out=None, eps=[-1.0, float("nan")])
    refused(fwd, ALIGN, b=F + 2, out=F + 1)
    refused(bwd, ARG, mean=None, rstd=None, dy=None, dx=None)
    refused(bwd, ALIGN, dy=F + 1, dx_out=F + 1, dx=F + 1, dw=F + 2, db=F + 1, ws=F + 4)
    refused(bwd, WORKSPACE, ws=None, size=[0, lib.oomb_layer_norm_workspace(4, 8) - 1])
    assert lib.oomb_layer_norm_workspace(1, 16385) == 0 and lib.oomb_layer_norm_workspace(0, 8) == 0


def test_head_loss_refusals(lib):
    def fwd(x=F, w=F, t=F, n=4, D=8, V=10, dtype=0, cap=0.0, loss=F, lse=F, ws=F, size=BIG, word=F):
        return lib.oomb_head_loss_fwd(x, w, t, n, D, V, dtype, cap, loss, lse, ws, size, word, None)

    def bwd(x=F, w=F, t=F, lse=F, d_loss=F, scale=1.0, n=4, D=8, V=10, dtype=0, cap=0.0, dx=F, dw=F, dw_dtype=0, acc=0,
            ws=F, size=BIG, word=F):
        return lib.oomb_head_loss_bwd(x, w, t, lse, d_loss, scale, n, D, V, dtype, cap, dx, dw, dw_dtype, acc, ws, size,
                                      word, None)

    inf, nan = float("inf"), float("nan")
    for call in (fwd, bwd):
        refused(call, ARG, x=None, w=None, t=None, lse=None, word=None, n=[0, -1], D=[0, -1], V=[0, -1, 2 ** 31 - 1],
                cap=[-1.0, nan, inf, 1e31, 1e-31])
        refused(call, DTYPE, dtype=2)
        refused(call, UNSUPPORTED, D=65537)
        refused(call, ALIGN, x=F + 1, w=F + 1, t=F + 4, lse=F + 2, ws=F + 16, word=F + 1)
        refused(call, WORKSPACE, ws=None, size=0)
    refused(fwd, ARG, loss=None)
    refused(fwd, ALIGN, loss=F + 2)
    refused(fwd, WORKSPACE, size=lib.oomb_head_loss_workspace(4, 8, 10, 0, 0) - 1)
    refused(bwd, ARG, scale=[inf, nan], acc=1)  # a bf16 gradient cannot be added to
    assert bwd(dx=None, dw=None) == ARG
    refused(bwd, DTYPE, dw_dtype=[2, -1])
    assert bwd(dtype=1, dw_dtype=0) == DTYPE  # fp32 operands, bf16 gradient
    refused(bwd, ALIGN, d_loss=F + 2, dx=F + 1, dw=F + 1)
    refused(bwd, WORKSPACE, size=lib.oomb_head_loss_workspace(4, 8, 10, 0, 1) - 1)
    for bad in ((0, 8, 10, 0), (4, 0, 10, 0), (4, 8, 0, 0), (4, 8, 10, 2), (4, 65537, 10, 0)):
        assert lib.oomb_head_loss_workspace(*bad, 1) == 0
    bits = C.c_uint32()
    assert lib.oomb_word_check(None, None, C.byref(bits)) == ARG and lib.oomb_word_check(F + 2, None, None) == ALIGN


def test_workspaces_serve_smaller_calls(lib):
    rows = [*range(1, 300), 513, 1000, 4097, 8192, 8193, 100000]
    for size in (lambda n: lib.oomb_embed_workspace(n, 100), lambda n: lib.oomb_layer_norm_workspace(n, 3584),
                 lambda n: lib.oomb_head_loss_workspace(n, 3584, 50001, 0, 0),
                 lambda n: lib.oomb_head_loss_workspace(n, 1000, 131072, 0, 1),
                 lambda n: lib.oomb_head_loss_workspace(n, 1001, 131072, 1, 1),
                 lambda n: lib.oomb_head_loss_workspace(n, 77, 77, 1, 0)):
        sizes = [size(n) for n in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for dt in (0, 1):
        assert lib.oomb_head_loss_workspace(100, 512, 9000, dt, 1) >= lib.oomb_head_loss_workspace(100, 512, 9000, dt, 0)


def test_python_calls_refuse_host_and_wrong_tensors(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t, tab, out, f = torch.zeros(4, dtype=torch.int64), torch.zeros(10, 8), torch.zeros(4, 8), torch.zeros(4)
    word = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        L.oomb_embed_fwd(t, tab, out, word)
    with pytest.raises(TypeError, match="int64"):
        L.oomb_embed_fwd(t.int(), tab, out, word)
    with pytest.raises(TypeError, match="unsupported dtype"):
        L.oomb_embed_fwd(t, tab.half(), out, word)
    with pytest.raises(ValueError, match="2 dimensions"):
        L.oomb_embed_bwd(t, out, tab[0], None, word)
    with pytest.raises(ValueError, match="current CUDA device"):
        L.oomb_layer_norm_fwd(out, None, None, out)
    with pytest.raises(ValueError, match="dimensions"):
        L.oomb_layer_norm_bwd(f, None, f, f, f, f)
    with pytest.raises(ValueError, match="current CUDA device"):
        L.oomb_head_loss_fwd(out, tab, t, f, f, None, word)
    with pytest.raises(TypeError, match="unsupported dtype"):
        L.oomb_head_loss_bwd(out.half(), tab, t, f, out, tab, None, word)
    with pytest.raises(TypeError, match="unsupported dtype"):
        L.oomb_head_loss_workspace(4, 8, 10, torch.float16, True)
    with pytest.raises(TypeError, match="32-bit"):
        L.oomb_word_check(t)
    with pytest.raises(ValueError, match="empty"):
        L.oomb_word_check(word[:0])


def test_model_ends_refusals():
    from paged_sparse_attention_gb300.ends import ModelEnds
    t = torch.zeros(10, 8)
    for kw, match in ((dict(head=torch.zeros(9, 8)), "one dtype"), (dict(head=t.bfloat16()), "one dtype"),
                      (dict(b_norm=torch.zeros(8)), "w_norm"), (dict(chunk=0), "positive")):
        with pytest.raises(ValueError, match=match):
            ModelEnds(t, **kw)
    with pytest.raises(ValueError, match="one dtype"):
        ModelEnds(t[0])
    ends = ModelEnds(t, chunk=4)  # (nothing runs before the first call)
    assert ends.d_head is ends.d_table and ends.ws.numel() > 0
