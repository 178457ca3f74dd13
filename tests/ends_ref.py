"""float64 values and error bounds of the operators at a model's two ends (CPU)."""
import torch

F64 = torch.float64
U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def head_reference(x, w, targets, cap=0.0, d_loss=None, scale=1.0, dw_dtype=None, grads=True):
    """Values and bounds of oomb_head_loss_fwd/bwd.

    A logit is a sum of D products in fp32, taken at least 16 at a step by the tensor cores (which may
    cut instead of round: 2^-23 of the largest partial sum a step) for up to 6 products of parts, or one
    at a step: (D + 32) 2^-24 times the sum of the products' magnitudes holds for both.  fp32 operands in
    three parts of 8 bits leave out products below 3 * 2^-24 of theirs: within the 32.  The exponent's
    argument is rounded in base 2 (2^-23 of its terms), the exponential is good to 2^-21, and its
    sum runs over at most 512 columns in a thread and V / 64 parts.  dz is rounded to x's type for bf16
    (fp32: three parts, 2^-23); a probability below fp32's least normal number is flushed to zero, an
    error of at most 2^-126; a product over K has K / 16 + 64 steps of 2^-23, in fp32 six times that.
    """
    n, D = x.shape
    V = w.shape[0]
    dt = x.dtype
    X, W = x.to(F64), w.to(F64)
    has = targets >= 0
    X = torch.where(has[:, None], X, torch.zeros((), dtype=F64))
    at = targets.clamp_min(0)
    z = X @ W.t()
    ez = (D + 32) * U32 * (X.abs() @ W.abs().t())
    t = None
    if cap > 0:
        t = torch.tanh(z / cap)
        ez = ez + cap * 2.0 ** -20 * t.abs()
        z = cap * t
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    e_exp = (z.abs() + lse.abs()[:, None]) * 2.0 ** -22 + 2.0 ** -21
    e_lse = ((p * (ez + e_exp)).sum(1) * 2 + (600 + V / 64) * U32 + 4 * U32 * lse.abs())
    rows = torch.arange(n)
    zt = z[rows, at]
    ref = {"lse": torch.where(has, lse, 0.0 * lse), "loss": torch.where(has, lse - zt, 0.0 * lse)}
    tol = {"lse": e_lse, "loss": e_lse + ez[rows, at] + 2 * U32 * (lse.abs() + zt.abs())}
    if not grads:
        return ref, tol
    g = torch.ones(n, dtype=F64) if d_loss is None else d_loss.to(F64)
    g = torch.where(has, g, 0.0 * g)
    q = p.clone()
    q[rows, at] -= 1.0
    eq = p * (ez + 2 * e_lse[:, None] + e_exp) * 1.01 + 2 * U32 * q.abs() + U32 * p + 2.0 ** -126
    dz = q
    if cap > 0:
        f = 1.0 - t * t
        eq = eq * f + q.abs() * 2 * t.abs() * (ez / cap + 4 * U32) + 4 * U32 * q.abs()
        dz = q * f
    dz, eq = dz * g[:, None], eq * g.abs()[:, None]
    eq = eq + dz.abs() * (half_step(torch.bfloat16) if dt == torch.bfloat16 else 2 * U32) + 2 * U32 * dz.abs()
    steps = 2 * (1 if dt == torch.bfloat16 else 6) * U32
    odt = dt if dw_dtype is None else dw_dtype
    ref["dx"] = scale * (dz @ W)
    tol["dx"] = abs(scale) * (eq @ W.abs() + (V / 16 + 64) * steps * (dz.abs() @ W.abs()))
    tol["dx"] += (half_step(dt) + 4 * U32) * ref["dx"].abs()
    ref["dw"] = scale * (dz.t() @ X)
    tol["dw"] = abs(scale) * (eq.t() @ X.abs() + (n / 16 + 64) * steps * (dz.abs().t() @ X.abs()))
    tol["dw"] += (half_step(odt) + 4 * U32) * ref["dw"].abs()
    return ref, tol


def check(out, ref, tol, names=None):
    for k in names or ref:
        got = out[k].cpu().to(F64)
        assert torch.isfinite(got).all(), k
        over = (got - ref[k]).abs() - tol[k]
        assert over.max().item() <= 0, (k, over.max().item(), tol[k].flatten()[over.argmax()].item())
