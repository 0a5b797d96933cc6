"""The checks of the orthogonalised update (update_ref.py) themselves, without a GPU: they let pass what the kernels' arithmetic gives,
and tell it from updates that are slightly wrong."""
import pytest
import torch

from tests import update_ref as ref

SIZES = [(1, 1), (1, 200), (200, 1), (2, 3), (5, 64), (63, 65), (64, 64), (65, 130), (128, 128), (129, 128), (127, 300), (150, 200), (257, 129),
         (200, 1000), (1000, 333), (256, 1024), (520, 512), (640, 2112), (64, 4096)]


def gradient(seed, n, k):
    gen = torch.Generator().manual_seed(seed)
    t = 2 * min(n, k) + 16
    return (torch.randn(t, n, generator=gen).t() @ torch.randn(t, k, generator=gen)).double() * 1e-3


def passes(out, limits):
    try:
        ref.check(out.to(torch.bfloat16), *limits)
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("n,k", SIZES)
def test_limits_of_a_gradient(n, k):
    g = gradient(n + k, n, k)
    a, b, c = ref.COEFFICIENTS
    limits = ref.limits(g)
    want = limits[0]
    for fp32 in (False, True):
        assert passes(ref.emulate(g, fp32=fp32), limits)
    assert passes(want, limits)
    last = want.clone()
    last[-1] = 0
    wrong = dict(zeros=0 * want, negated=-want, larger=1.02 * want, smaller=0.98 * want, last=last, four=ref.exact(g, steps=4),
                 six=ref.exact(g, steps=6), b=ref.exact(g, coefficients=(a, 1.02 * b, c)), c=ref.exact(g, coefficients=(a, b, 0.95 * c)))
    if min(n, k) > 4:
        wrong["bf16"] = ref.emulate(g, kept=torch.bfloat16)
    assert [name for name, out in wrong.items() if passes(out, limits)] == []


@pytest.mark.parametrize("n,k", [(40, 60), (300, 900), (1000, 640)])
@pytest.mark.parametrize("name", ref.PRODUCTS)
def test_limits_of_a_product(n, k, name):
    """A product that is missing, has the wrong sign, is 2% off, misses a K step, or has one tile of zeros."""
    coefficients, steps, _ = ref.PRODUCTS[name]
    g, u, v = ref.of_rank(3, n, k, [1.0] * ref.RANK)
    how = dict(steps=steps, coefficients=coefficients, scale=ref.product_scale(name))
    limits = ref.product_limits(name, u, v)
    want = limits[0]
    for fp32 in (False, True):
        assert passes(ref.emulate(g, fp32=fp32, **how), limits)
    tile = want.clone()
    tile[-30:, -30:] = 0
    short = (u if n <= k else v).clone()        # of A = X X^T, the smaller side's
    long = v if n <= k else u
    lost = long[64:].t() @ long[64:] if max(n, k) > 64 else torch.zeros(8, 8, dtype=torch.float64)
    wrong = dict(zeros=0 * want, negated=-want, larger=1.02 * want, tile=tile)
    if name == "A X":
        x = short @ lost @ long.t()
        wrong["lost"] = x if n <= k else x.t()
    assert [w for w, out in wrong.items() if passes(out, limits)] == []
