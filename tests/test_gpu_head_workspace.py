"""The forward of the loss over a vocabulary by itself, in a workspace of its own size: values, and nothing written
behind it."""
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
@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("n,V,D", [(8192, 100, 64), (9728, 100, 64), (3840, 300, 64), (3584, 300, 72), (3000, 260, 65),
                                   (512, 2400, 64), (800, 1100, 200), (336, 2316, 64), (19456, 33, 64), (19457, 33, 64),
                                   (33, 4800, 64), (70, 9001, 136), (300, 40961, 64), (20, 70000, 520), (3, 5000, 64)])
def test_forward_in_a_workspace_of_its_own(dtype, off, n, V, D):
    x, w, t, _ = make(n, V, D, dtype, seed=n + V, masked=0.02)
    wc = torch.empty(w.numel() + off, dtype=dtype, device="cuda")[off:].view(V, D).copy_(w)
    size = L.oomb_head_loss_workspace(n, D, V, dtype, False)
    space = torch.full((size + (1 << 18),), 171, dtype=torch.uint8, device="cuda")
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    err = word()
    L.oomb_head_loss_fwd(x.cuda(), wc, t.cuda(), loss, lse, space[:size], err)
    assert L.oomb_word_check(err) == 0
    assert (space[size:] == 171).all()
    check({"loss": loss, "lse": lse}, *head_reference(x, w, t, grads=False))


def test_calls_of_every_size_in_the_workspace_of_the_longest():
    """Fewer rows go another way and still stay inside."""
    V, D = 300, 64
    size = L.oomb_head_loss_workspace(3900, D, V, BF, False)
    space = torch.full((size + (1 << 18),), 171, dtype=torch.uint8, device="cuda")
    for n in (1, 8, 9, 255, 256, 257, 1024, 3583, 3840, 3841, 3900):
        x, w, t, _ = make(n, V, D, BF, seed=n)
        loss, lse, err = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), word()
        L.oomb_head_loss_fwd(x.cuda(), w.cuda(), t.cuda(), loss, lse, space[:size], err)
        assert L.oomb_word_check(err) == 0
        assert (space[size:] == 171).all()
        check({"loss": loss, "lse": lse}, *head_reference(x, w, t, grads=False))
