"""Rotary positions of any size: angles against 60-digit arithmetic."""
import math
import struct
from decimal import Decimal as D
from decimal import getcontext

import numpy as np
import pytest
import torch

import paged_sparse_attention_gb300 as L

pytestmark = pytest.mark.gpu

getcontext().prec = 60
TWO_PI = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


FAR = [0, 1, -1, 12345, -(1 << 22), (1 << 30) + 7, -(1 << 40) - 1, (1 << 40) + 3, (1 << 50) + 12345, -(1 << 53) - 1,
       (1 << 62) - 999, (1 << 63) - 1, -(1 << 63)]


@pytest.mark.parametrize("theta", [1e4, 1e6, 1.5])
@pytest.mark.parametrize("d,axes,own_ladder", [(128, 2, False), (80, 3, True), (10, 1, True), (2, 1, False)])
@pytest.mark.parametrize("mode", [1, 2])
def test_angles_of_far_positions(theta, d, axes, own_ladder, mode):
    half, n, H = d // 2, len(FAR), 2
    axis = [j % axes for j in range(half)]
    pos = [[(p * (a + 1) + (1 << 63)) % (1 << 64) - (1 << 63) for p in FAR] for a in range(axes)]
    x = torch.randn(n, H, d, generator=torch.Generator().manual_seed(d))
    out = torch.full_like(x, float("nan")).cuda()
    L.oomb_bias_rope_axes(x.cuda(), None, out, H, torch.tensor(pos).cuda(), axis, theta, mode, own_ladder=own_ladder)
    ln = D(struct.unpack("f", struct.pack("f", theta))[0]).ln()
    z = x.double().numpy()
    ref, seen = np.empty_like(z), [0] * axes
    for j, a in enumerate(axis):
        e = D(seen[a]) / axis.count(a) if own_ladder else D(j) / half
        seen[a] += 1
        freq = (-ln * e).exp() / TWO_PI
        ang = np.array([float((p * freq) % 1) for p in pos[a]]) * 2 * math.pi * (1 if mode == 1 else -1)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        ref[..., j], ref[..., j + half] = z[..., j] * c - z[..., j + half] * s, z[..., j + half] * c + z[..., j] * s
    # the angle: 2^-26 turns as a float and 2^-31 before; cos and sin: two half steps of values up
    # to 1; then two products and a sum, half a step each
    mag = np.abs(z[..., :half]) + np.abs(z[..., half:])
    tol = np.concatenate([mag, mag], -1) * (2 * math.pi * (2.0 ** -26 + 2.0 ** -31) + 2 * 2.0 ** -24 + 3 * 2.0 ** -24)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()
