"""The feed-forward operators with tensors past 2^32 bytes: inputs made of one small block over and over, whose outputs
are the small run's, bit for bit, wherever they lie; and two graphs that share a memory pool."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests.gpu_util import device
from tests.test_gpu_ffn import experts, rand, routing

pytestmark = pytest.mark.gpu


def repeated(block, times):
    """[times * len(block), ...] of one block."""
    out = torch.empty((times * block.shape[0], *block.shape[1:]), dtype=block.dtype, device=block.device)
    out.view(times, *block.shape)[:] = block
    return out


def same_blocks(big, small, dim=0):
    parts = big.split(small.shape[dim], dim)
    return all(torch.equal(parts[i], small) for i in (0, len(parts) // 2, len(parts) - 1))


@pytest.mark.parametrize("M,tile", [(20, None), (20, "128x128"), (300, "256x288")])
def test_linear_weight_past_32_bits(M, tile, monkeypatch):
    if tile:
        monkeypatch.setenv("FG_GEMM_TILE", tile)
    N, K, times = 5632, 131072, 6
    xq, sx = fg.fg_quantize_act_1x128(rand(1, M, K))
    wq = torch.randint(0, 0x70, (N, K), dtype=torch.uint8, device=device(), generator=torch.Generator(device()).manual_seed(1))
    sw = torch.rand(N // 128, K // 128, device=device(), generator=torch.Generator(device()).manual_seed(2)) + 0.5
    small = fg.fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, act=fg.FG_ACT_RELU, out_dtype=torch.float32)
    big = fg.fg_fp8_gemm_fprop_epilogue(xq, sx, repeated(wq, times), repeated(sw, times), act=fg.FG_ACT_RELU, out_dtype=torch.float32)
    assert bool(torch.isfinite(small).all()) and same_blocks(big, small, 1)


def test_act_forward_past_32_bits():
    F, times = 16384, 140
    z = rand(1, 1000, 2 * F)
    small = fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_SILU, gated=True)
    big = fg.fg_act_checkpoint_fwd(repeated(z, times), fg.FG_ACT_SILU, gated=True)
    for a, b, dim in zip(big, small, (0, 1, 0, 1)):
        assert same_blocks(a, b, dim)


def test_act_backward_past_32_bits():
    F, times = 16384, 1094
    zq, sz = fg.fg_quantize_act_1x128(rand(1, 128, 2 * F))
    da = rand(2, 128, F, dtype=torch.float32)
    small = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_SILU, gated=True, bias_grad=True)
    big = fg.fg_act_checkpoint_bwd(repeated(zq, times), sz.repeat(1, times), repeated(da, times), fg.FG_ACT_SILU, gated=True, bias_grad=True)
    for a, b, dim in zip(big[:6], small[:6], (0, 1, 1, 0, 1, 0)):
        assert same_blocks(a, b, dim)
    # 1094 equal addends: at most 18 of a wave in turn, four at a time, and 16 waves (every addition half a step off)
    want = small.dbias.double() * times
    assert bool(((big.dbias.double() - want).abs() <= (times / 16 + 1 + 16) * 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("T", [5, 40])
def test_moe_weights_past_32_bits(T):
    E, H, I = 48, 8192, 8192
    one = experts(1, 1, H, I)
    x = rand(2, T, H)
    ids, weights = routing(3, T, 1, 1, 1)
    small = fg.fg_moe_few_tokens(x, ids, weights, *one)
    big = [repeated(w, E) for w in one]
    for e in (0, 31, E - 1):
        assert torch.equal(fg.fg_moe_few_tokens(x, ids + e, weights, *big), small), e


def test_two_graphs_of_one_pool():
    """Two captures that share a pool (their workspaces lie in the same memory), replayed in turn with eager work between."""
    we = experts(7, 8, 512, 256)
    x = rand(1, 48, 512)
    ids, weights = routing(2, 48, 4, 8, 8)
    zq, sz = fg.fg_quantize_act_1x128(rand(3, 512, 512))
    da = rand(4, 512, 256, dtype=torch.float32)

    def first():
        return (fg.fg_moe_few_tokens(x, ids, weights, *we), fg.fg_moe_few_tokens(x[:9], ids[:9], weights[:9], *we))

    def second():
        r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_GELU_TANH, gated=True, bias_grad=True)
        return (*r, fg.fg_moe_few_tokens(x[8:40], ids[8:40], weights[8:40], *we))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first(), second()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        outs = [first()]
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        outs.append(second())
    for k in range(4):
        x.copy_(rand(10 + k, 48, 512))
        da.copy_(rand(20 + k, 512, 256, dtype=torch.float32))
        for graph, out, eager in zip(graphs, outs, (first, second)):
            graph.replay()
            want = eager()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), k
