"""Calls of the feed-forward operators that their documentation allows or refuses, beside the sizes of test_gpu_ffn.py."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests.gpu_util import device
from tests.test_gpu_ffn import check_linear, check_moe, experts, linear_case, rand, routing

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


@pytest.mark.parametrize("M,N,K", [(4097, 64, 1024), (5000, 17, 640), (8192, 130, 512), (20001, 8, 1152), (16384, 200, 128),
                                   (70001, 3, 256), (65535 * 16, 1, 128), (65535 * 16 + 1, 1, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_many_rows_on_a_narrow_weight(M, N, K, dtype):
    """A router's projection in training: more rows than 4096 on a few columns."""
    ops = linear_case(M, M, N, K)
    bias, residual = rand(1, N), rand(2, M, N, dtype=dtype)
    y = torch.full((M, N), float("nan"), dtype=dtype, device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_SILU, residual=residual, y=y)
    check_linear(ops, y, "silu", bias, residual)


@pytest.mark.parametrize("T", [1, 2, 9, 16])
@pytest.mark.parametrize("H,I,E,topk", [(4096, 128, 3, 2), (4224, 256, 4, 3), (5120, 1152, 4, 4), (8192, 384, 2, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_moe_wide_layers_for_few_tokens(T, H, I, E, topk, dtype):
    """From 4096 columns on the down-projection has two 16-column tiles a workgroup and is not split."""
    w = experts(H + E, E, H, I)
    x = rand(T, T, H)
    ids, weights = routing(T + H, T, topk, E + 1, E)
    y = fg.fg_moe_few_tokens(x, ids, weights, *w, out_dtype=dtype)
    check_moe(y, (x, ids, weights, *w), "silu", False)


@pytest.mark.parametrize("M,N,tile", [(5000, 64, None), (5000, 300, None), (4096, 2048, None), (300, 200, "128x128"), (300, 200, "256x192"),
                                      (300, 200, "256x256"), (300, 200, "256x288")])
def test_linear_empty_contraction_of_many_rows_and_on_tiles(M, N, tile, monkeypatch):
    if tile:
        monkeypatch.setenv("FG_GEMM_TILE", tile)
    ops = linear_case(1, M, N, 0)
    bias, residual = rand(1, N), rand(2, M, N)
    y = torch.full((M, N), float("nan"), device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_GELU_TANH, residual=residual, y=y)
    check_linear(ops, y, "gelu", bias, residual)


def test_linear_activations_past_32_bits():
    """A few columns of more than 2^32 bytes of activations: the first, middle and last rows against 64 bits."""
    M, N, K = 70000, 8, 65536
    g = torch.Generator(device()).manual_seed(1)
    xq = torch.randint(0, 0x70, (M, K), dtype=torch.uint8, device=device(), generator=g)
    wq = torch.randint(0, 0x70, (N, K), dtype=torch.uint8, device=device(), generator=g)
    sx = torch.rand(K // 128, M, device=device(), generator=g) + 0.5
    sw = torch.rand(1, K // 128, device=device(), generator=g) + 0.5
    y = fg.fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, out_dtype=torch.float32)
    for rows in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
        check_linear((xq[rows], sx[:, rows].contiguous(), wq, sw), y[rows], "none", None, None)
