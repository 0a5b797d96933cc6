"""The orthogonalised update on the GPU within limits that follow from its fp16 roundings (update_ref.py): whole updates, each product
of a step by itself on every tile, and spectra other than that of independent tokens."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests import update_ref as ref
from tests.gpu_util import device
from tests.test_gpu_train import SIDES, T, dirty_workspace, gradient

pytestmark = pytest.mark.gpu


def update(g, **how):
    """The update of a matrix or batch, into a buffer and workspace that hold something else."""
    shape = g.shape if g.dim() == 3 else (1, *g.shape)
    return fg.fg_orthogonalize(g, out=torch.full(g.shape, float("nan"), dtype=torch.bfloat16, device=device()),
                               workspace=dirty_workspace(*shape), **how)


@pytest.mark.parametrize("n,k", SIDES)
@pytest.mark.parametrize("dtype", ["f", "b"])
def test_sizes(n, k, dtype):
    g = gradient(n + k, n, k, T[dtype])
    ref.check(update(g, scale=0.5), *ref.limits(g.double(), scale=0.5), (n, k))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_steps(steps):
    g = gradient(3, 150, 200)
    ref.check(update(g, steps=steps), *ref.limits(g.double(), steps=steps), steps)


@pytest.mark.parametrize("batch,n,k", [(1, 64, 8192), (2, 76, 16200), (3, 5000, 130), (4, 60, 4200), (1, 309, 4853), (1, 700, 8192),
                                       (1, 856, 11323), (2, 1024, 8192), (1, 2048, 16384), (1, 2000, 18000), (1, 8200, 1500), (1, 1500, 1300),
                                       (1, 2001, 1000), (8, 512, 1024), (4, 1024, 4096), (1, 2560, 2560), (1, 4096, 4160), (8, 2000, 2040),
                                       (8, 2048, 7168), (1, 7168, 18432)])
def test_large(batch, n, k):
    """Five steps on every tile, the rest of a round and shared contractions."""
    g = torch.stack([gradient(i, n, k) for i in range(batch)])
    out = update(g)
    for i in {0, batch // 2, batch - 1}:
        ref.check(out[i], *ref.limits(g[i].double()), (n, k, i))


# ---- each product by itself -----------------------------------------------------------------------------

TILES = [(1, 40, 60), (1, 300, 900), (1, 64, 8192), (2, 76, 16200), (1, 856, 11323), (1, 1000, 2001), (1, 1100, 4200), (1, 2040, 2100), (3, 1030, 2100),
         (1, 4096, 4160), (8, 2048, 2048), (9, 2050, 1990), (1, 2048, 8448), (8, 2000, 2040), (8, 512, 1024), (8, 1024, 2050), (1, 2000, 10400),
         (8, 2048, 7168), (8, 2000, 7000), (1, 1536, 16384), (1, 2000, 18000), (1, 3000, 18432), (1, 4096, 4096), (1, 7168, 18432), (1, 18432, 7168)]


@pytest.mark.parametrize("batch,n,k", TILES)
@pytest.mark.parametrize("name", ref.PRODUCTS)
def test_products(batch, n, k, name):
    """A step of one term and eight equal directions, so that the result is that product alone."""
    coefficients, steps, _ = ref.PRODUCTS[name]
    made = [ref.of_rank(100 * i + n, n, k, [1.0] * ref.RANK, torch.float32, device()) for i in range(batch)]
    out = update(torch.stack([m[0] for m in made]), steps=steps, coefficients=coefficients, scale=ref.product_scale(name))
    for i in {0, batch // 2, batch - 1}:
        ref.check(out[i], *ref.product_limits(name, *made[i][1:]), (batch, n, k, i))


# ---- spectra --------------------------------------------------------------------------------------------

def spectrum(name, m):
    i = torch.arange(1, m + 1, dtype=torch.float64)
    return {"1/sqrt i": i ** -0.5, "1/i": 1 / i, "1/i^2": i ** -2, "exp(-i/20)": torch.exp(-i / 20), "exp(-i/100)": torch.exp(-i / 100),
            "flat": torch.ones_like(i)}[name]


# what the header states of the update before it is rounded to bf16
SPECTRA = {"flat": 2e-3, "1/sqrt i": 2e-3, "1/i": 4.5e-3, "1/i^2": 2.5e-2, "exp(-i/20)": 1.5e-2, "exp(-i/100)": 6.5e-3}


@pytest.mark.parametrize("name", SPECTRA)
@pytest.mark.parametrize("n,k", [(128, 512), (512, 1024), (2048, 1024)])
def test_spectra(name, n, k):
    g = ref.of_rank(5, n, k, spectrum(name, min(n, k)), torch.float32, device())[0]
    limits = ref.limits(g.double())
    out = update(g)
    ref.check(out, *limits, name)
    want = limits[0]
    assert float((out.double() - want).norm() / want.norm()) <= (SPECTRA[name] ** 2 + 2e-3 ** 2) ** 0.5


@pytest.mark.parametrize("rank,stated", [(1, 0.15), (4, 0.08), (16, 0.05), (64, 0.03), (256, 0.009)])
def test_few_directions(rank, stated):
    """Along its directions the update is p^5(s), and the raised roundings in its empty ones are as large as the header says, within
    a tenth."""
    n, k = 1000, 1400
    g, u, v = ref.of_rank(7, n, k, [1.0] * rank, torch.float32, device())
    out = update(g).double()
    limits = ref.limits(g.double())
    ref.check(out, *limits, rank)
    want = limits[0]
    assert float((out - want).norm() / want.norm()) <= 1.1 * stated + 2e-3
    along = (u * (out @ v)).sum(0)                  # u^T out v of each direction
    s = rank ** -0.5
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    # X, A and B round each element by itself, which hardly moves a direction as a whole: what the header says of ordinary gradients
    assert float((along - s).abs().max()) <= 1.6e-3, (along, s)


@pytest.mark.parametrize("size,stated", [(1e-10, 2e-3), (1e-12, 2e-3), (1e-13, 3e-3), (1e-14, 3e-2)])
def test_far_below_eps(size, stated):
    """Gradients far smaller than eps (1e-7), whose X has entries that fp16 holds with fewer bits."""
    g = gradient(5, 256, 1024)
    g *= size / g.double().norm()
    limits = ref.limits(g.double())
    out = update(g)
    ref.check(out, *limits, size)
    want = limits[0]
    assert float((out.double() - want).norm() / want.norm()) <= (stated ** 2 + 2e-3 ** 2) ** 0.5


@pytest.mark.parametrize("eps", [1.5e-45, 1e-41, 2.9e-39, 3e-39, 1e-30])
def test_zeros_of_any_eps(eps):
    assert not update(torch.zeros(70, 90, device=device()), eps=eps).any()
    assert not update(torch.zeros(90, 70, device=device(), dtype=torch.bfloat16), eps=eps).any()


@pytest.mark.parametrize("size,eps", [(1e-40, 1e-43), (3e-39, 1e-45), (2e-38, 1e-41), (1e-41, 2e-38), (1e-37, 1e-37), (1e30, 1e-45), (3e38, 1e-7), (3e38, 3e38),
                                      (1e38, 3.3e38)])
@pytest.mark.parametrize("n,k", [(120, 200), (200, 120)])
def test_ends_of_fp32(size, eps, n, k):
    """|G| and eps whose sum is denormal or past fp32's range, although X is neither."""
    g = gradient(6, n, k).double()
    g = (g * (size / float(g.norm()))).float()
    eps = float(torch.tensor(eps, dtype=torch.float32))
    ref.check(update(g, eps=eps), *ref.limits(g.double(), eps=eps), (size, eps))


@pytest.mark.parametrize("scale", [1e-31, -1e-36, 1e-37, 3e-38, 1e38, -0.0])
@pytest.mark.parametrize("n,k", [(8, 8), (500, 300), (1100, 4200), (2048, 8448)])
def test_scales(n, k, scale):
    """Factors whose product with X's and B's own scales is denormal, on each kind of tile: the same numbers times the factor, as
    long as those are not denormal themselves. One direction of eight ones, so that they are 1 / 8 and 0."""
    g = torch.zeros(n, k, device=device())
    g[:8, :8] = 1
    one = update(g, steps=1, coefficients=(1.0, 0.0, 0.0))
    out = update(g, steps=1, coefficients=(1.0, 0.0, 0.0), scale=scale)
    want = torch.zeros(n, k, dtype=torch.float64, device=device())
    want[:8, :8] = 0.125
    assert torch.equal(one.double(), want)
    tiny = 2.0 ** -134 if abs(scale) < 1e-37 else 0.0           # half a step of a denormal bf16
    factor = float(torch.tensor(scale, dtype=torch.float32))
    assert bool(((out.double() - factor * want).abs() <= (factor * want).abs() * 2.0 ** -8 + tiny).all())
