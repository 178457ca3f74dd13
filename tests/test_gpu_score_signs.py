"""Attention with modified scores under negative scales and slopes, where a maximum of the raw
products is no maximum of the scores: -q and -scale give the scores of q and scale."""
import pytest
import torch

import paged_sparse_attention_gb300 as L
from score_ref import check
from test_gpu_score_attn import SHAPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (0.0, -1.0), (20.0, 0.0), (20.0, -1.0), (0.0, 30.0)])
@pytest.mark.parametrize("mask", ["causal", "empty", "prefix"])
@pytest.mark.parametrize("shape", ["tc_g2_ragged", "tc_few_tokens_inside", "fp32_64", "bf16_odd_page"])
def test_negative_scale(shape, mask, cap, slope):
    c = Case(cap=cap, bias=slope != 0.0, mask=mask, sel="all", seed=9, spread=2.0, **SHAPES[shape])
    if slope:
        c.slopes = c.slopes * slope
        c.mod["slopes"] = c.slopes.cuda()
    q = c.q
    c.q = -q
    ref = c.reference()
    c.q, c.scale = q, -c.scale
    ref["dq"] = -ref["dq"]
    o, lse = c.forward()
    dq = c.backward(o, lse)
    assert L.oomb_check(c.pool.handle) == 0
    dk, dv = c.pool.logical_grads(c.total)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, x, ref)
    c.pool.close()
