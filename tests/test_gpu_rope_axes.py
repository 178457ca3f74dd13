"""Rotary positions with several axes on the GPU against float64 complex numbers."""
import numpy as np
import pytest
import torch

import paged_sparse_attention_gb300 as L

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_sparse_attention_gb300 import build
    build.build()
    L.load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def turned(x, bias, positions, axis, theta, mode, own_ladder):
    n, H, d = x.shape
    half = d // 2
    z = x.double().numpy() + (0 if bias is None else bias.double().numpy().reshape(1, H, d))
    if mode == 0:
        return z
    axis = np.asarray(axis)
    expo = np.arange(half) / half
    if own_ladder:
        for a in set(axis.tolist()):
            i = np.flatnonzero(axis == a)
            expo[i] = np.arange(i.size) / i.size
    ang = positions.numpy()[axis].T.astype(np.float64) * np.power(float(theta), -expo)
    w = (z[..., :half] + 1j * z[..., half:]) * np.exp((1j if mode == 1 else -1j) * ang)[:, None]
    return np.concatenate([w.real, w.imag], -1)


def call(x, bias, positions, axis, theta, mode, own_ladder, out_dtype):
    out = torch.full(x.shape, float("nan"), dtype=out_dtype, device="cuda")
    L.oomb_bias_rope_axes(x.cuda(), None if bias is None else bias.cuda(), out, x.shape[1],
                          None if positions is None else positions.cuda(), axis, theta, mode, own_ladder=own_ladder)
    return out


def check(got, ref, x, bias, out_dtype, positions):
    """The fp32 steps: the angle is known to 2^-31 turns; cos and sin are off by at most 2^-22;
    two products and a sum; then one rounding.  Far positions: the factor goes through three
    roundings of 2^-53 here and the reference's angle through two."""
    n, H, d = x.shape
    half = d // 2
    z = x.double().abs().numpy() + (0 if bias is None else bias.double().abs().numpy().reshape(1, H, d))
    mag = z[..., :half] + z[..., half:]
    far = 0.0 if positions is None else float(positions.abs().max()) * 5 * 2.0 ** -53
    tol = (2.0 ** -21 + 2 * np.pi * 2.0 ** -31 + far) * np.concatenate([mag, mag], -1) + \
        torch.finfo(out_dtype).eps / 2 * np.abs(ref)
    err = np.abs(got.double().cpu().numpy() - ref) - tol
    assert np.isfinite(got.float().cpu().numpy()).all() and err.max() <= 0, err.max()


@pytest.mark.parametrize("ti,to", [(FP, BF), (BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("H,d,n", [(28, 128, 65), (3, 80, 33), (1, 2, 5), (5, 24, 1), (4, 64, 700), (2, 10, 129)])
@pytest.mark.parametrize("mode,own_ladder", [(1, False), (2, True), (0, False)])
def test_rotation_matches(ti, to, H, d, n, mode, own_ladder):
    g = torch.Generator().manual_seed(d * n)
    x = torch.randn(n, H, d, generator=g).to(ti)
    bias = torch.randn(H * d, generator=g) if mode == 1 else None
    A = min(3, d // 2)
    axis = [j % A for j in range(d // 2)] if not own_ladder else [min(A - 1, j * A // (d // 2)) for j in range(d // 2)]
    pos = torch.randint(-1000, 5_000_000, (A, n), generator=g)
    ref = turned(x, bias, pos, axis, 1e6, mode, own_ladder)
    check(call(x, bias, pos, axis, 1e6, mode, own_ladder, to), ref, x, bias, to, pos)


def test_one_axis_is_the_plain_rotation():
    """Positions in one axis, all pairs on it: bias_rope's rotation, far into a sequence."""
    g = torch.Generator().manual_seed(2)
    n, H, d, pos0 = 100, 4, 128, 4_194_304 - 100
    x, bias = torch.randn(n, H, d, generator=g), torch.randn(H * d, generator=g)
    pos = torch.arange(pos0, pos0 + n)[None].contiguous()
    y = torch.empty(n, H, d, device="cuda")
    for mode in (1, 2):
        L.oomb_bias_rope(x.cuda(), bias.cuda(), y, H, pos0, 1e6, mode)
        a = call(x, bias, pos, [0] * 64, 1e6, mode, False, FP)
        check(y, turned(x, bias, pos, [0] * 64, 1e6, mode, False), x, bias, FP, pos)
        check(a, turned(x, bias, pos, [0] * 64, 1e6, mode, False), x, bias, FP, pos)


def test_far_positions_in_place_and_back():
    """Positions of 2^40, the rotation in place, and the inverse undoing it."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(16, 2, 64, generator=g)
    axis = [1] * 32  # an axis may go unused
    pos = torch.stack([torch.zeros(16, dtype=torch.int64), (1 << 40) + torch.arange(16)])
    ref = turned(x, None, pos, axis, 1e4, 1, False)
    y = x.cuda()
    L.oomb_bias_rope_axes(y, None, y, 2, pos.cuda(), axis, 1e4, 1)
    check(y, ref, x, None, FP, pos)
    L.oomb_bias_rope_axes(y, None, y, 2, pos.cuda(), axis, 1e4, 2)
    assert (y.cpu() - x).abs().max().item() < 2.0 ** -19 * 8  # two turns, 2^-21 of at most |x| + |y| each


def test_rows_off_16_bytes():
    g = torch.Generator().manual_seed(7)
    x = torch.randn(9, 2, 64, generator=g).to(BF)
    buf = torch.empty(x.numel() + 1, dtype=BF, device="cuda")
    buf[1:] = x.view(-1).cuda()
    pos = torch.arange(9)[None].contiguous()
    out = torch.empty(x.numel() + 1, device="cuda")[1:].view(x.shape)
    L.oomb_bias_rope_axes(buf[1:].view(x.shape), None, out, 2, pos.cuda(), [0] * 32, 1e4, 1)
    check(out, turned(x, None, pos, [0] * 32, 1e4, 1, False), x, None, FP, pos)


def test_refusals():
    x = torch.zeros(4, 2, 8, device="cuda")
    o = torch.empty_like(x)
    pos = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    ok = [0, 1, 0, 1]
    bad = [
        (ValueError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos, [0, 1, 0], 1e4, 1)),       # pairs
        (ValueError, lambda: L.oomb_bias_rope_axes(x, None, o, 3, pos, ok, 1e4, 1)),              # heads
        (ValueError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos[:, :3], ok, 1e4, 1)),       # positions
        (TypeError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos.int(), ok, 1e4, 1)),
        (ValueError, lambda: L.oomb_bias_rope_axes(x.cpu(), None, o, 2, pos, ok, 1e4, 1)),
        (ValueError, lambda: L.oomb_bias_rope_axes(x[..., ::2], None, o[..., ::2], 2, pos, [0, 1], 1e4, 1)),
        (TypeError, lambda: L.oomb_bias_rope_axes(x.half(), None, o, 2, pos, ok, 1e4, 1)),
        (L.OombError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos, [0, 1, 2, 0], 1e4, 1)),   # axis
        (L.OombError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos, ok, 1.0, 1)),             # theta
        (L.OombError, lambda: L.oomb_bias_rope_axes(x, None, o, 2, pos, ok, 1e4, 3)),             # mode
    ]
    for kind, f in bad:
        with pytest.raises(kind):
            f()


def test_offsets_past_32_bits():
    """More than 2^31 elements, in place: the last tokens get what a call of their own gives them."""
    n, H, d, last = 600500, 28, 128, 40
    x = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(last, H, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    x[-last:] = tail
    pos = torch.arange(2 * n, device="cuda").view(2, n)
    axes = bytes(j % 2 for j in range(d // 2))
    want = torch.empty_like(tail)
    L.oomb_bias_rope_axes(tail, None, want, H, pos[:, -last:].contiguous(), axes, 1e6, 1)
    L.oomb_bias_rope_axes(x, None, x, H, pos, axes, 1e6, 1)
    assert torch.equal(x[-last:], want) and not x[-last - 1].any()


@pytest.mark.parametrize("axes", [[0, 1] * 4, torch.tensor([0, 1] * 4), bytearray([0, 1] * 4)])
def test_axes_as_any_sequence(axes):
    x = torch.randn(5, 2, 16, generator=torch.Generator().manual_seed(4)).cuda()
    pos = torch.arange(10, device="cuda").view(2, 5)
    a, b = torch.empty_like(x), torch.empty_like(x)
    L.oomb_bias_rope_axes(x, None, a, 2, pos, bytes([0, 1] * 4), 1e4, 1)
    L.oomb_bias_rope_axes(x, None, b, 2, pos, axes, 1e4, 1)
    assert torch.equal(a, b)
    with pytest.raises(TypeError):  # a number of axes is not a list of them
        L.oomb_bias_rope_axes(x, None, b, 2, pos, 8, 1e4, 1)
