"""A block norm whose wait for a row runs out (the first row's copy is never started; the wait is
bounded): the status, sums that say so themselves, and a GPU that goes on."""
import pytest
import torch

import paged_sparse_attention_gb300 as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def inputs(dtype, n, D, gate):
    g = torch.Generator(device="cuda").manual_seed(n + D)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {k: rn(n, D).to(dtype) for k in ("x", "y", "du", "dx_out")}
    t.update(w_pre=1 + 0.1 * rn(D), w_post=1 + 0.1 * rn(D))
    t["gate"] = {"channel": lambda: rn(D), "token": lambda: rn(n, D).to(dtype)}[gate]()
    return t


def run(t, backward):
    n, D = t["x"].shape
    par = {k: t[k] for k in ("w_pre", "w_post", "gate")}
    r = [torch.empty(n, device="cuda") for _ in range(2)]
    xo, u = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    L.oomb_block_norm_fwd(t["x"], t["y"], xo, u, rstd_pre=r[0], rstd_post=r[1], **par)
    if not backward:
        return lambda: L.oomb_block_norm_fwd(t["x"], t["y"], xo, u, rstd_pre=r[0], rstd_post=r[1], **par), [xo, u]
    dx, dy = torch.empty_like(xo), torch.empty_like(xo)
    dw = [torch.empty(D, device="cuda") for _ in range(2)]
    ws = torch.empty(L.oomb_block_norm_workspace(n, D), dtype=torch.uint8, device="cuda")
    return lambda: L.oomb_block_norm_bwd(t["x"], t["y"], dx, dy, du=t["du"], dx_out=t["dx_out"], rstd_pre=r[0],
                                         rstd_post=r[1], dw_pre=dw[0], dw_post=dw[1], workspace=ws,
                                         **par), [dx, dy, *dw]


# rows that stay in registers from their load, rows whose stage goes back late, odd widths
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype,n,D,gate", [(torch.bfloat16, 8192, 3584, "channel"), (torch.bfloat16, 8192, 3584, "token"),
                                            (torch.bfloat16, 4096, 8192, "channel"), (torch.float32, 4097, 1537, "token")])
def test_a_wait_that_runs_out_is_reported(dtype, n, D, gate, backward):
    call, out = run(inputs(dtype, n, D, gate), backward)
    call()
    assert L.oomb_block_norm_check() == 0
    want = [t.clone() for t in out]
    L.oomb_block_norm_test_timeout(True)
    try:
        call()
    finally:
        L.oomb_block_norm_test_timeout(False)
    with pytest.raises(L.OombError) as e:
        L.oomb_block_norm_check()
    assert e.value.status == 6  # TIMEOUT
    if backward:
        assert all(torch.isnan(t).all() for t in out[2:])
    assert L.oomb_block_norm_check() == 0  # read once
    call()
    assert L.oomb_block_norm_check() == 0
    for a, b in zip(out, want):
        assert torch.equal(a, b)
