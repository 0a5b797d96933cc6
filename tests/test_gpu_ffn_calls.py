"""Calls of the feed-forward operators that their documentation allows or refuses, beside the sizes of test_gpu_ffn.py."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests.gpu_util import device
from tests.test_gpu_ffn import experts, rand, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("H", [1, 8, 16, 31, 32, 100, 127, 129, 200])
@pytest.mark.parametrize("given", [False, True])
def test_moe_width_that_is_no_multiple_of_a_tile_is_refused(T, H, given):
    """Narrower than a column block too; with and without a workspace of the caller's."""
    _, s1, w2, s2 = experts(1, 2, 128, 128)
    ids, weights = routing(1, T, 1, 2, 2)
    w1 = torch.zeros(2, 256, H, dtype=torch.uint8, device=device())
    w2 = torch.zeros(2, H, 128, dtype=torch.uint8, device=device())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=device()) if given else None
    with pytest.raises(fg.Fp8fgError, match="shape"):
        fg.fg_moe_few_tokens(rand(2, T, H), ids, weights, w1, s1, w2, s2, workspace=ws)
    assert fg.lib().fg_last_hip_error() == 0
