"""Plain statements in 64 bits of the feed-forward operators, and checks of FP8 codes against real values."""
import math

import torch

EPS24 = 2.0 ** -24                # half a step of fp32, relative
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}    # max |act'|


def act(z, kind):
    """(act(z), act'(z)) of a float64 tensor."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return torch.relu(z), (z > 0).double()
    if kind == "silu":
        k = torch.special.expit(z)
        return z * k, k * (1 + z * (1 - k))
    a = math.sqrt(2 / math.pi)
    th = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th ** 2) * a * (1 + 3 * 0.044715 * z ** 2)


def decode(q):
    return q.view(torch.float8_e4m3fn).float().double()


def rows_values(q, s):
    """Codes [r, c] with scales [c / 128, r] (tiles along the columns) -> float64 values."""
    return decode(q) * s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def block_values(q, s):
    """Codes [n, k] with scales [ceil(n / 128), k / 128] -> float64 values."""
    return decode(q) * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)


def scale_of(amax, pow2):
    """The scale rule of include/fp8fg.h on float64 max-abs values; also float64, but held in 32 bits."""
    s = (amax / 448).float().double().clamp(min=2.0 ** -126)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    return torch.where(amax == 0, torch.ones_like(s), s)


def grid_step(q):
    """Distance between neighbouring E4M3 values around |q|."""
    _, e = torch.frexp(q.abs().clamp(max=448))
    return torch.ldexp(torch.ones_like(q), (e - 1).clamp(min=-6) - 3)


def grid(q):
    step = grid_step(q)
    return (torch.round(q / step) * step).clamp(-448, 448)


def check_tiles(q, s, v, err, pow2, what):
    """Codes q [r, c] and scales s [c / 128, r] against the real values v, which the kernel had within err (a tensor
    like v): each scale follows from a max-abs within err of the real one, and each code is a nearest one of a
    quotient within err of the real one, by the scale that was written (half a step; the quotient itself is
    rounded to 32 bits)."""
    r, c = v.shape
    vt, et = v.unflatten(1, (-1, 128)), err.unflatten(1, (-1, 128))
    s = s.double().t()                                                   # [r, c / 128]
    lo = (vt.abs() - et).clamp(min=0).amax(2)
    hi = (vt.abs() + et).amax(2)
    assert s.shape == lo.shape, (what, s.shape, lo.shape)
    s_lo, s_hi = scale_of(lo, pow2), scale_of(hi, pow2)
    if pow2:
        assert bool(((s == s_lo) | (s == s_hi)).all()), what
    else:
        zero = hi == 0
        # a max-abs that may be 0 may also be any small value, whose scale goes down to the smallest one
        s_lo = torch.where(lo == 0, torch.full_like(lo, 2.0 ** -126), s_lo)
        ok = torch.where(zero, s == 1, (s >= s_lo * (1 - 2 * EPS24)) & (s <= s_hi * (1 + 2 * EPS24)) | (lo == 0) & (s == 1))
        assert bool(ok.all()), (what, (s / s_lo - 1).abs().max(), (s / s_hi - 1).abs().max())
    quot = vt / s[:, :, None]
    d = decode(q).unflatten(1, (-1, 128))
    step = grid_step(torch.maximum(quot.abs(), d.abs()))
    far = (d - quot).abs() - (step / 2 + et / s[:, :, None] + 2 * EPS24 * quot.abs())
    assert float(far.max()) <= 0, (what, float(far.max()))


def grad_error(z, kind):
    """Bound on the error of act and act' in fp32, for the kernel's sigmoid k: exp(-z) is off by (|z| + 4) 2^-24
    relative (the rounded product with log2(e), and one unit of 2^x), k by that and two roundings, and act' =
    k + a (1 - k) [2 u'] sums terms of at most 1 + |z| (GELU: k (1 - k) z^3 stays below that too) with each
    factor's relative error and a rounding; z itself was rounded to 32 bits, and |act''| < 1.2."""
    if kind in ("none", "relu"):
        return 2 * EPS24 * (1 + z.abs())
    return (4 * z.abs() + 32) * EPS24 * (1 + z.abs())


def moe(x, ids, weights, w1q, s1, w2q, s2, kind, pow2, gate=1e-3):
    """(y, bound): the layer in 64 bits, and how far a kernel may be from it whose products of FP8 codes are within
    `gate` of the largest of the row (the GEMMs' own limit for fp32 outputs). A hidden value within that
    error of a border between two codes may get the other one; one away from borders may not."""
    T, H = x.shape
    E, I = w1q.shape[0], w2q.shape[2]
    t = x.double().unflatten(1, (-1, 128))
    s = scale_of(t.abs().amax(2), pow2)
    xv = (grid((t / s[:, :, None]).float().double()) * s[:, :, None]).flatten(1)
    y, bound = torch.zeros_like(xv), torch.zeros_like(xv)
    for e in range(E):
        hit = ids == e
        rows = hit.any(1).nonzero()[:, 0]
        if not len(rows):
            continue
        share = (weights.double() * hit).sum(1)[rows, None]
        w1, w2 = block_values(w1q[e], s1[e]), block_values(w2q[e], s2[e])
        gu = xv[rows] @ w1.t()
        err = gate * gu.abs().amax(1, keepdim=True)
        g, u = gu[:, :I], gu[:, I:]
        a = act(g, kind)[0]
        h = a * u
        he = LIPSCHITZ[kind] * err * (u.abs() + err) + a.abs() * err + grad_error(g, kind) * u.abs()
        ht, et = h.unflatten(1, (-1, 128)), he.unflatten(1, (-1, 128))
        s = scale_of(ht.abs().amax(2), pow2)[:, :, None]
        lo = scale_of((ht.abs() - et).clamp(min=0).amax(2), pow2)[:, :, None]
        hi = scale_of((ht.abs() + et).amax(2), pow2)[:, :, None]
        q = ht / s
        hv = grid(q.float().double()) * s
        if pow2:        # the neighbour's scale, where the max-abs may reach it, is another grid altogether
            other = torch.where((lo != s) | (hi != s), grid_step(q) * s * 2, torch.zeros_like(hv))
            move = et
        else:
            other = torch.zeros_like(hv)
            move = et + ht.abs() * ((hi - lo) / s)
        step = grid_step(q)
        border = (q / step - torch.floor(q / step) - 0.5).abs() * step * s      # distance to the tie
        flip = torch.where(border <= move * 1.01, step * s, torch.zeros_like(hv))
        he = (flip + other + (0 if pow2 else 1) * hv.abs() * ((hi - lo) / s)).flatten(1)
        y[rows] += share * (hv.flatten(1) @ w2.t())
        out = hv.flatten(1) @ w2.t()
        bound[rows] += share.abs() * (he @ w2.abs().t() + gate * out.abs().amax(1, keepdim=True))
    return y, bound
