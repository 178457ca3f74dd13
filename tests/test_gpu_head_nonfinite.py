"""Logits that overflow: a row whose softmax is no number says so, and the rows beside it keep their values."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from ends_ref import check, head_reference
from test_gpu_head_loss import make, word

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [6, 20, 300])
@pytest.mark.parametrize("at_target", [True, False])
def test_an_overflowing_logit(dtype, n, at_target):
    """One logit of row 2 is +infinity, its target's or another's: inf - inf, or an infinite loss, and never a small one."""
    V, D = 500, 64
    x, w, t, _ = make(n, V, D, dtype, seed=n)
    x[:, 0] = 0.0
    w[:, 0] = 0.0
    t[2], loud = 7, 7 if at_target else 400
    w[loud, 0] = 4.0
    big = x.clone()
    big[2, 0] = 2e38
    out, err = {k: torch.zeros(n, device="cuda") for k in ("loss", "lse")}, word()
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, dtype, False), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(big.cuda(), w.cuda(), t.cuda(), out["loss"], out["lse"], ws, err)
    assert L.oomb_word_check(err) == 0
    assert not torch.isfinite(out["loss"][2]) and not torch.isfinite(out["lse"][2])
    rest = torch.arange(n) != 2
    ref, tol = head_reference(x[rest], w, t[rest], grads=False)
    check({k: v[rest.cuda()] for k, v in out.items()}, ref, tol)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [6, 300])
def test_a_target_of_minus_infinity(dtype, n):
    """Its probability is 0: an infinite loss, and the sum of the others as it is."""
    V, D = 500, 64
    x, w, t, _ = make(n, V, D, dtype, seed=n + 1)
    x[:, 0] = 0.0
    w[:, 0] = 0.0
    t[2] = 7
    w[7, 0] = -4.0
    big = x.clone()
    big[2, 0] = 2e38
    out, err = {k: torch.zeros(n, device="cuda") for k in ("loss", "lse")}, word()
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, dtype, False), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(big.cuda(), w.cuda(), t.cuda(), out["loss"], out["lse"], ws, err)
    assert L.oomb_word_check(err) == 0
    assert out["loss"][2] == float("inf")
    ref, tol = head_reference(torch.cat([x[2:3]]), torch.cat([w[:7], w[8:]]), torch.tensor([0]), grads=False)
    assert abs(float(out["lse"][2]) - float(ref["lse"][0])) <= float(tol["lse"][0])
