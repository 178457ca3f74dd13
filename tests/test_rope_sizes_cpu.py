"""Sizes that the multi-axis rotation refuses, on the CPU (placeholder pointers)."""
import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300 import build

F = 1 << 24  # a placeholder address


def test_a_token_past_32_bits_is_refused():
    build.build()
    lib = L.load()
    for mode in (0, 1):
        for H, d in ((1 << 25, 64), (1 << 30, 2), ((1 << 24) + 1, 128)):
            assert H * d >= 1 << 31
            assert lib.oomb_bias_rope_axes(F, 0, None, F, 0, 1, H, d, F, 1, bytes(d // 2), 1e4, 0, mode, None) == 8
