"""The orthogonalised update on the GPU within limits that follow from its fp16 roundings (update_ref.py): whole updates, and each
product of a step by itself on every tile."""
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
