"""What LayerStep.run takes as a chunk's dO, from a tensor or from a function: only what the kernels can read."""
import pytest
import torch

from paged_sparse_attention_gb300.layer import chunk_gradient


def test_a_chunk_gradient_is_like_the_output():
    o = torch.zeros(6, 2, 4, dtype=torch.bfloat16)
    for good in (torch.ones_like(o), torch.ones(6, 8, dtype=torch.bfloat16), torch.ones(12, 2, 4, dtype=torch.bfloat16)[6:]):
        assert chunk_gradient(good, o) is good
    with pytest.raises(TypeError, match="bfloat16, not torch.float32"):
        chunk_gradient(torch.ones(6, 2, 4), o)
    with pytest.raises(TypeError, match="NoneType"):
        chunk_gradient(None, o)
    for few in (torch.ones_like(o)[:5], torch.ones(6, 2, 5, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="needs"):
            chunk_gradient(few, o)
    one = torch.ones((), dtype=torch.bfloat16)
    for laid in (one.expand(6, 2, 4), torch.ones(2, 6, 4, dtype=torch.bfloat16).transpose(0, 1)):
        with pytest.raises(ValueError, match="contiguous"):
            chunk_gradient(laid, o)
    with pytest.raises(ValueError, match="meta"):
        chunk_gradient(torch.ones(6, 2, 4, dtype=torch.bfloat16, device="meta"), o)
