"""LayerStep.run with a function in place of dO: it is asked once a chunk, last first, and what it returns is checked."""
import pytest
import torch

from paged_sparse_attention_gb300.layer import LayerStep
from paged_sparse_attention_gb300.pool import PagedKVPool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_function_for_the_gradient(dtype):
    from paged_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Hq, Hkv, d, P, N, Dm = 2, 1, 64, 64, 200, 96
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev)  # noqa: E731
    W = [rn(Dm, H * d) * 0.1 for H in (Hq, Hkv, Hkv)]
    layer = LayerStep(PagedKVPool(Hq, Hkv, d, P, 4, 4, dtype, dev), *W, chunk=128)
    X, dO, asked = rn(N, Dm), rn(N, Hq, d), []

    def part(start, o):
        asked.append((start, tuple(o.shape)))
        return dO[start:start + o.shape[0]]

    want, got = layer.run(X, dO), layer.run(X, part)
    assert asked == [(128, (72, Hq, d)), (0, (128, Hq, d))]
    for k in ("dX", "dWq", "dWk", "dWv"):
        assert torch.equal(want[k], got[k]), k
    one = torch.ones((), dtype=dtype, device=dev)
    for bad, error in ((lambda s, o: one.expand_as(o), ValueError), (lambda s, o: torch.ones_like(o)[1:], ValueError),
                       (lambda s, o: torch.ones_like(o).cpu(), ValueError), (lambda s, o: None, TypeError),
                       (lambda s, o: torch.ones_like(o).half(), TypeError)):
        with pytest.raises(error):
            layer.run(X, bad)
    with pytest.raises(ValueError, match="contiguous"):
        layer.run(X, rn(N, d, Hq).transpose(1, 2))
    assert torch.equal(layer.run(X, dO)["dX"], want["dX"])
