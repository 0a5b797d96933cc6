"""What the orthogonalised update's fp16 operands leave of it: the kernels' roundings emulated around sums in 64 bits, and checks
whose limits follow from those."""
import torch

from tests.train_ref import COEFFICIENTS

SCALE_X, SCALE_A = 4096.0, 2048.0


def _wide(g):
    return (g, False) if g.shape[0] <= g.shape[1] else (g.t().contiguous(), True)


def exact(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7, scale=1.0):
    """The update of one float64 matrix, in 64 bits."""
    a, b, c = coefficients
    x, tall = _wide(g)
    x = x / (torch.linalg.matrix_norm(x) + eps)
    for _ in range(steps):
        p = x @ x.t()
        q = b * p + c * (p @ p)
        q.diagonal().add_(a)
        x = q @ x
    return scale * (x.t() if tall else x)


def emulate(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7, scale=1.0, kept=torch.float16, fp32=False, nudge=None):
    """The same with X, A and B = a I + b A + c A A rounded to `kept` where the kernels round them, X times 2^12 and A and B times
    2^11, and sums in 64 bits, or with `fp32` in 32. Not rounded to bf16 at the end. `nudge`: a generator that moves each
    value by 2^-16 up or down first."""
    a, b, c = coefficients
    x, tall = _wide(g)

    def r(v):
        if nudge is not None:
            v = v * (1 + 2.0 ** -16 * torch.randint(-1, 2, v.shape, generator=nudge).to(v.device))
        return v.to(kept).double()

    def product(p, q):
        return (p.float() @ q.float()).double() if fp32 else p @ q
    x = r(x / (torch.linalg.matrix_norm(x) + eps) * SCALE_X)
    for s in range(steps):
        p = r(product(x, x.t()) * (SCALE_A / SCALE_X ** 2))
        q = c / SCALE_A * product(p, p) + b * p
        q.diagonal().add_(a * SCALE_A)
        y = product(r(q), x)
        x = r(y / SCALE_A) if s + 1 < steps else y * (scale / (SCALE_A * SCALE_X))
    return x.t() if tall else x


def limits(g, **how):
    """(update, limit in the 2-norm, limits of its elements) for a bf16 output. The store's rounding is known. What X, A and B
    lose is twice what the emulation of the same gradient loses: fp32 sums in another order take a rounding to the neighbouring
    value now and then, after which later roundings are others of the same size, and a sum of several hundred of those is
    near its usual size (at 20 sizes emulated with 32-bit sums, 0.9 to 1.1 times). Sides of one and two have too few of them for that, but
    their sums, of up to 200 squares, are within 200 half steps (2^-16.4): there it is the most that any of 32 emulations loses whose
    values were moved by about that before they were rounded."""
    want, emulated = exact(g, **how), emulate(g, **how)
    if min(g.shape) <= 2:
        gen = torch.Generator().manual_seed(1)
        moved = [emulate(g, nudge=gen, **how) for _ in range(32)]
        off = torch.stack([m - want for m in moved]).abs().max(0).values
        return want, max(float((m.to(torch.bfloat16).double() - want).norm()) for m in moved), want.abs() * 2.0 ** -8 + 1.01 * off
    store, off = (want.to(torch.bfloat16).double() - want).norm(), 2 * (emulated - want).abs()
    return want, float((store.square() + off.norm().square()).sqrt()), want.abs() * 2.0 ** -8 + 1.01 * off.max()


def check(out, want, limit, element, what=""):
    """An update within its limits. (1.02: bf16 steps of what is off by its fp16 roundings instead of the exact value's.)"""
    off = (out.double() - want).abs()
    assert bool(torch.isfinite(out).all()), what
    assert float(off.norm()) <= 1.02 * limit, (what, float(off.norm() / want.norm()), limit / float(want.norm()))
    assert bool((off <= element).all()), (what, float((off - element).max()))


def of_rank(seed, n, k, singular, dtype=torch.float64, device="cpu"):
    """(matrix, U, V) with these singular values and random directions."""
    gen = torch.Generator().manual_seed(seed)
    r = len(singular)
    u, v = (torch.linalg.qr(torch.randn(d, r, generator=gen, dtype=torch.float64))[0].to(device) for d in (n, k))
    s = torch.as_tensor(singular, dtype=torch.float64, device=device)
    return ((u * s) @ v.t()).to(dtype), u, v


# A step of one term: coefficients, steps, and the number of half steps (2^-11) that fp16 takes of the result, to first order: X as
# often as it is a factor, A as often as it is, and B; with two steps the X between them too.
PRODUCTS = {"X": ((1.0, 0.0, 0.0), 1, 2), "X twice": ((1.25, 0.0, 0.0), 2, 4), "A X": ((0.0, 2.0, 0.0), 1, 5), "A A X": ((0.0, 0.0, 2.0), 1, 8)}
RANK = 8


def product_scale(name):
    """What makes the result of a matrix of RANK equal directions U V^T."""
    coefficients, steps, _ = PRODUCTS[name]
    value = RANK ** -0.5
    for _ in range(steps):
        value = sum(c * value ** e for c, e in zip(coefficients, (1, 3, 5)))
    return 1 / value


def product_limits(name, u, v):
    """As `limits`, for the result U V^T. Half a step of a factor's every element changes an element (i, j) of the result by no more than
    half a step of |U_i| |V_j|."""
    want = u @ v.t()
    store, off = (want.to(torch.bfloat16).double() - want).norm(), PRODUCTS[name][2] * 2.0 ** -11
    element = 1.02 * (want.abs() * 2.0 ** -8 + off * u.norm(dim=1)[:, None] * v.norm(dim=1)[None])
    return want, float((store.square() + RANK * off ** 2).sqrt()), element
