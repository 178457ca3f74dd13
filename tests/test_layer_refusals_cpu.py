"""Calls that the layer step refuses before anything runs (no GPU: the weights' cast is left out)."""
import types

import pytest
import torch

from paged_sparse_attention_gb300 import layer


@pytest.fixture
def make(monkeypatch):
    def no_launch(*a, **k):
        raise AssertionError("a refused call has reached the library")

    def build(**kw):
        pool = types.SimpleNamespace(Hq=2, Hkv=1, d=8, P=4, dtype=torch.float32, device=torch.device("cpu"), handle=0,
                                     workspace=no_launch)
        monkeypatch.setattr(layer.L, "oomb_bias_rope", lambda *a, **k: None)
        step = layer.LayerStep(pool, torch.zeros(6, 16), torch.zeros(6, 8), torch.zeros(6, 8), chunk=4,
                               gemm_workspace_bytes=16, **kw)
        monkeypatch.setattr(layer.L, "oomb_pool_reset", no_launch)
        return step

    return build


X, DO = torch.zeros(8, 6), torch.zeros(8, 2, 8)
DOCS = torch.tensor([0, 3, 8])


@pytest.mark.parametrize("kw", [dict(top_k=0), dict(top_k=2), dict(top_k=2, n_sink=0), dict(window=3),
                                dict(window=0, n_sink=2)])
def test_documents_with_a_selection_that_does_not_know_them(make, kw):
    with pytest.raises(ValueError, match="documents"):
        make(**kw).run(X, DO, doc_start=DOCS)


@pytest.mark.parametrize("kw,run", [(dict(top_k=-1), {}), (dict(window=3, n_sink=0), {}),
                                    (dict(top_k=2), dict(sel_override=[None, None])), (dict(top_k=2), None)])
def test_what_goes_with_documents(make, kw, run):
    """Every page, a window without sinks, given pages, or no documents: not refused (the next call is reached)."""
    args = {} if run is None else dict(doc_start=DOCS, **run)
    with pytest.raises(AssertionError, match="reached the library"):
        make(**kw).run(X, DO, **args)


def test_prefixes_that_cross_a_chunk():
    """Against the rows themselves: a row of the prefix' document sees less than the prefix."""
    g = torch.Generator().manual_seed(3)
    for _ in range(300):
        chunk, n = int(torch.randint(1, 9, (1,), generator=g)), int(torch.randint(1, 40, (1,), generator=g))
        cuts = torch.randint(-5, n + 6, (5,), generator=g).sort().values
        pre = torch.randint(-3, 20, (4,), generator=g)
        want = []
        for c in range(4):
            a, b = int(cuts[c]), int(cuts[c + 1])
            end = min(a + int(pre[c]), b, n)  # the prefix, as far as there are tokens
            rows = range(max(a, 0), min(b, n))
            want.append(any(min(end, (i // chunk + 1) * chunk) < end for i in rows))
        assert layer.prefix_cut(cuts, pre, chunk, n).tolist() == want, (chunk, n, cuts, pre)


def test_nothing_of_a_call_is_kept(make):
    step = make(softcap=3.0)
    with pytest.raises(AssertionError):
        step.run(X, DO, doc_start=DOCS)
    assert step._docs is None and step._positions is None and step._ws_fwd is None
