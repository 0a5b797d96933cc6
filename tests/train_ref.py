"""Plain statements in 64 bits of the training step's norm and orthogonalised update, with bounds on fp32 and fp16 rounding."""
import math

import torch

from tests.ffn_ref import EPS24

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def norm(x, gamma, beta, layer, eps):
    """(y, bound of its fp32 error, mean, its bound, rstd, its relative bound). A row's sums pass through at most 24 additions in
    a thread, 6 in its wave and 16 over the waves, so a sum is off by 46 roundings of the sum of magnitudes. That makes the
    mean's bound; the squares' sum, whose terms are positive and have two roundings each, is off by 48 relative, the mean's own
    error adds its square, and the root halves both; division by n, + eps, root and reciprocal round once more each."""
    n = x.shape[1]
    mean = x.mean(1) if layer else torch.zeros(x.shape[0], dtype=x.dtype, device=x.device)
    mean_err = 48 * EPS24 * x.abs().sum(1) / n if layer else torch.zeros_like(mean)
    d = x - mean[:, None]
    var = d.square().mean(1) + eps
    rstd = var ** -0.5
    rel = 30 * EPS24 + mean_err.square() / var
    h = d * rstd[:, None]
    h_err = rstd[:, None] * (EPS24 * d.abs() + mean_err[:, None]) + h.abs() * (rel[:, None] + EPS24)
    y = h * gamma + (0 if beta is None else beta)
    return y, gamma.abs() * h_err + EPS24 * ((h * gamma).abs() + y.abs()), mean, mean_err, rstd, rel


def norm_grad(x, mean, rstd, gamma, dy, dres, layer):
    """(dx, bound before it is stored, dgamma, dbeta, sum of |dy xhat|, sum of |dy|), with mean and rstd as they are."""
    n = x.shape[1]
    d = x - mean[:, None] if layer else x
    h = d * rstd[:, None]
    h_err = 2 * EPS24 * h.abs()
    t = dy * gamma
    t1 = t.mean(1, keepdim=True) if layer else torch.zeros_like(t[:, :1])
    t2 = (t * h).mean(1, keepdim=True)
    t1_err = 50 * EPS24 * t.abs().mean(1, keepdim=True) if layer else 0.0
    t2_err = 52 * EPS24 * (t * h).abs().mean(1, keepdim=True)
    dx = (t - t1 - h * t2) * rstd[:, None]
    err = rstd[:, None] * (3 * EPS24 * (t.abs() + t1.abs() + (h * t2).abs()) + t1_err + h.abs() * t2_err + t2.abs() * h_err)
    err = err + EPS24 * dx.abs()
    if dres is not None:
        dx = dx + dres
        err = err + EPS24 * dx.abs()
    return dx, err, (dy * h).sum(0), dy.sum(0), (dy * h).abs().sum(0), dy.abs().sum(0)


def largest_singular(gram):
    """Square root of the largest eigenvalue, of large matrices by powers (and 2% more, for what they miss)."""
    if gram.shape[0] <= 700:
        return float(torch.linalg.matrix_norm(gram, 2)) ** 0.5
    v = torch.ones(gram.shape[0], 1, dtype=gram.dtype, device=gram.device) + torch.arange(gram.shape[0], device=gram.device)[:, None] % 7
    for _ in range(100):
        v = gram @ (v / v.norm())
    return 1.02 * float(v.norm()) ** 0.5


def orthogonalize(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7, scale=1.0):
    """(update, bound of the fp16 roundings in the 2-norm) of one float64 matrix. To first order a step p(X) = a X + b X X^T X + c
    (X X^T)^2 X takes a change of X to one no larger than the largest |p'| on [0, u] times it, u its largest singular value; a
    step's own roundings (half a step, 2^-11 relative, of X, A and B = a I + b A + c A A) enter it as 2^-11 (L |X| + (|b| |A|
    + 2 |c| |A| u^2 + |B|) u)."""
    a, b, c = coefficients
    x = g if g.shape[0] <= g.shape[1] else g.t()
    x = x / (torch.linalg.matrix_norm(x) + eps)
    half, err = 2.0 ** -11, 0.0
    for _ in range(steps):
        p = x @ x.t()
        u = largest_singular(p)
        s = torch.linspace(0, u, 1001, dtype=torch.float64)
        slope = float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max())
        q = b * p + c * (p @ p)
        q.diagonal().add_(a)
        fro = [float(torch.linalg.matrix_norm(v)) for v in (x, p, q)]
        err = slope * err + half * (slope * fro[0] + (abs(b) * fro[1] + 2 * abs(c) * fro[1] * u * u + fro[2]) * u)
        x = q @ x
    x = x if g.shape[0] <= g.shape[1] else x.t()
    return scale * x, abs(scale) * err


def check_update(out, want, err, what=""):
    """Against the exact update: the 2-norm within the bound (and the store's own rounding), and no element further off than six
    times what the bound makes evenly spread over the matrix."""
    want = want.to(out.device)
    assert bool(torch.isfinite(out).all()), what
    off = out.double() - want
    store = want.abs() * 2.0 ** -8
    assert float(off.norm()) <= 1.1 * err + float(store.norm()), (what, float(off.norm()), err)
    spread = 6 * 1.1 * err / math.sqrt(want.numel())
    if want.numel() > 256:
        far = float((off.abs() - store * 1.05 - spread).max())
        assert far <= 0, (what, far)
