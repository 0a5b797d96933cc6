"""The norm's values at the ends of fp32's range, on the GPU."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests.gpu_util import device
from tests.test_gpu_train import check_norm, rand, rows_like

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,weight,eps", [(1e15, 1e24, 1e-5), (1e-3, 1e36, 1e-5), (1e15, 1e-30, 1e-5), (1e-17, 1e-28, 1e-38), (1e16, 3e35, 1e-44)])
@pytest.mark.parametrize("rows,cols,tokens", [(3, 512, False), (300, 2304, False), (128, 640, True)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gamma_of_any_size(size, weight, eps, rows, cols, tokens, kind):
    """x gamma leaves fp32's range or has few bits there, although y is an ordinary number."""
    x = rows_like(1, rows, cols, torch.float32) * size
    gamma, beta = (1 + rand(2, cols, std=0.2)) * weight, rand(3, cols, std=0.1) * weight
    for b in (None, beta):
        r = fg.fg_norm_quantize(x, gamma, b, kind=fg.FG_NORM_LAYER if kind == "layer" else fg.FG_NORM_RMS, eps=eps, token_tiles=tokens, with_y=True)
        assert bool(torch.isfinite(r.y).all())
        check_norm(r, x, gamma, b, kind == "layer", float(torch.tensor(eps, dtype=torch.float32)), False, (size, weight))


@pytest.mark.parametrize("value", [2.0 ** 70, -(2.0 ** 110), 2.0 ** -120])
@pytest.mark.parametrize("rows,cols,tokens", [(3, 512, False), (300, 2048, False), (128, 1024, True)])
def test_constant_rows_and_a_tiny_eps(value, rows, cols, tokens):
    """x - mean is zero and rstd 1 / sqrt(eps), whose product with the mean is past fp32's range: y is beta."""
    x = torch.full((rows, cols), value, device=device())
    gamma, beta = 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    for b in (None, beta):
        r = fg.fg_norm_quantize(x, gamma, b, eps=1e-44, token_tiles=tokens, with_y=True)
        assert bool((r.mean == value).all())
        check_norm(r, x, gamma, b, True, float(torch.tensor(1e-44, dtype=torch.float32)), False, value)
        assert torch.equal(r.y, (0 * gamma if b is None else b).to(torch.bfloat16).expand(rows, cols))
