"""oomb_doc_spans with as many rows as an int holds."""
import pytest
import torch

import paged_sparse_attention_gb300 as L

pytestmark = pytest.mark.gpu


def test_rows_up_to_the_largest_int():
    from paged_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = (1 << 31) - 1
    cuts = torch.tensor([0, 5, n - 3, 1 << 40], device="cuda")
    b, e = (torch.full((n + 8,), -1, dtype=torch.int64, device="cuda") for _ in range(2))
    L.oomb_doc_spans(cuts, 0, b[:n], e[:n])
    assert b[:6].tolist() == [0, 0, 0, 0, 0, 5] and e[:6].tolist() == [1, 2, 3, 4, 5, 6]
    assert b[n - 5:].tolist() == [5, 5, n - 3, n - 3, n - 3] + [-1] * 8
    assert e[n - 5:].tolist() == [n - 4, n - 3, n - 2, n - 1, n] + [-1] * 8
    assert bool((e[:n] > b[:n]).all())
