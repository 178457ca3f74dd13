"""Long sums of one sign in the gradients of the loss over a vocabulary: nothing is lost that grows with their length."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
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


def flat(n, V, D, dtype, dw_dtype, base=None):
    """dw of logits that are all 0 under targets that are all 0, for weights g of eight bits: every column behind the
    first has dz = g / V, V a power of two, which bf16 holds, and so the gradient sum(g x) / V, whose terms are all
    positive."""
    x = torch.rand(n, D, generator=torch.Generator("cuda").manual_seed(n), device="cuda")
    x = x.mul_(torch.linspace(0, 1, D, device="cuda")).add_(1.0).to(dtype)  # another sum in each column
    g = 1.0 + torch.randint(0, 128, (n,), device="cuda") / 128
    w = torch.zeros(V, D, dtype=dtype, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, lse, err = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), word()
    dw = torch.full((V, D), float("nan"), dtype=dw_dtype, device="cuda") if base is None else base.clone()
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, dtype, True), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(x, w, t, loss, lse, ws, err)
    L.oomb_head_loss_bwd(x, w, t, lse, None, dw, ws, err, d_loss=g, accumulate=base is not None)
    assert L.oomb_word_check(err) == 0
    return dw[1:].to(F64), (x.to(F64) * g[:, None]).sum(0) / V


# The tensor cores add 16 products at a step and cut the sum there, at most twice by 2^-23 of it.  A piece of 28 steps
# of 64 rows has 112 such steps, at which its sum of equal signs is half of what it becomes on the average; the n / 1792
# pieces are added in fp32, 2^-24 each of at most the whole; the scale, the old value and the store are three more.
def cuts(n):
    return (112 + n / 1792 / 2 + 2) * 2.0 ** -23


@pytest.mark.parametrize("n", [9000, 65536])
@pytest.mark.parametrize("added", [False, True])
def test_fp32_gradient_of_bf16_operands(n, added):
    V, D = 4096, 768
    base = torch.rand(V, D, device="cuda") if added else None
    got, want = flat(n, V, D, BF, FP, base)
    if added:
        want = base[1:].to(F64) + want
    assert ((got - want).abs() <= cuts(n) * want).all(), float(((got - want).abs() / want).max())


def test_fp32_gradient_of_fp32_operands():
    """An exponential that is off by up to 2^-20 is not rounded to a power of two here."""
    got, want = flat(20000, 4096, 768, FP, FP)
    assert ((got - want).abs() <= (cuts(20000) + 2.0 ** -20) * want).all(), float(((got - want).abs() / want).max())


def test_bf16_gradient_of_very_many_rows():
    n = 262144
    got, want = flat(n, 1024, 2560, BF, BF)
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want).exponent - 9)  # of a step of bf16 at this value
    assert ((got - want).abs() <= half + cuts(n) * want).all(), float((((got - want).abs() - half) / want).max())


@pytest.mark.parametrize("D", [8192, 65536])
@pytest.mark.parametrize("dw_dtype", [BF, FP])
def test_probabilities_of_wide_rows(D, dw_dtype):
    """Every logit of a row is the same long sum of one sign: each probability is 1 / V, a power of two, unless the backward
    forms other logits than the forward did.  (Off by less than 2^-9 it is rounded to 1 / V.)"""
    n, V = 300, 2048
    x = torch.rand(n, D, generator=torch.Generator("cuda").manual_seed(D), device="cuda").add_(1.0).to(BF)
    w = torch.full((V, D), 213 / 128 * 2.0 ** -10 * 65536 / D, dtype=BF, device="cuda")  # logits of about 160
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, lse, err = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), word()
    dw = torch.full((V, D), float("nan"), dtype=dw_dtype, device="cuda")
    ws = torch.empty(L.oomb_head_loss_workspace(n, D, V, BF, True), dtype=torch.uint8, device="cuda")
    L.oomb_head_loss_fwd(x, w, t, loss, lse, ws, err)
    L.oomb_head_loss_bwd(x, w, t, lse, None, dw, ws, err)
    assert L.oomb_word_check(err) == 0
    want = x.to(F64).sum(0) / V
    tol = cuts(n) + (torch.finfo(BF).eps / 2 if dw_dtype is BF else 0.0)
    assert ((dw[1:].to(F64) - want).abs() <= tol * want).all(), float(((dw[1:].to(F64) - want).abs() / want).max())
