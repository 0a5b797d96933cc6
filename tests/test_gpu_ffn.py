"""The feed-forward operators on the GPU against their definitions in 64 bits: the Linear with its epilogue, the
activation with its FP8 checkpoint and its backward, and the mixture of experts for a few tokens."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests import ffn_ref as ref
from tests.gpu_util import TOL_F32, device

pytestmark = pytest.mark.gpu


def rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(device())


def act_code(kind):
    return ref.ACTS[kind]


# ---- Linear with its epilogue -------------------------------------------------------------------------

def linear_case(seed, M, N, K, pow2=False):
    x, w = rand(seed, M, K), rand(seed + 1, N, K, std=0.5 * max(K, 1) ** -0.5)
    if K == 0:
        return (torch.empty((M, 0), dtype=torch.uint8, device=device()), torch.empty((0, M), device=device()),
                torch.empty((N, 0), dtype=torch.uint8, device=device()), torch.empty(((N + 127) // 128, 0), device=device()))
    return (*fg.fg_quantize_act_1x128(x, pow2=pow2), *fg.fg_quantize_w_128x128(w, pow2=pow2))


def check_linear(ops, y, kind, bias, residual):
    xq, sx, wq, sw = ops
    z = ref.rows_values(xq, sx) @ ref.block_values(wq, sw).t()
    # the GEMMs' limit on an fp32 sum, through an activation of bounded slope
    gemm = TOL_F32 * float(z.abs().max()) if z.numel() else 0.0
    if bias is not None:
        z = z + bias.double()
    want = ref.act(z, kind)[0]
    tol = ref.LIPSCHITZ[kind] * (gemm + ref.EPS24 * z.abs()) + ref.grad_error(z, kind)
    if residual is not None:
        want = want + residual.double()
    tol = tol + ref.EPS24 * want.abs()
    if y.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    assert bool(torch.isfinite(y).all())
    far = ((y.double() - want).abs() - tol)
    assert float(far.max()) <= 0, float(far.max())


SHAPES = [(1, 1, 128), (1, 16, 256), (1, 1000, 1024), (3, 17, 128), (16, 130, 640), (17, 129, 256), (33, 65, 1280),
          (64, 256, 384), (65, 300, 256), (100, 77, 512), (128, 192, 256), (257, 259, 384), (300, 2001, 256),
          (512, 1024, 1024)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("pow2", [False, True])
def test_linear_shapes(M, N, K, pow2):
    ops = linear_case(M * 7 + N, M, N, K, pow2)
    bias, residual = rand(5, N, dtype=torch.float32), rand(6, M, N)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_SILU, residual=residual, y=y, pow2=pow2)
    check_linear(ops, y, "silu", bias, residual)


@pytest.mark.parametrize("M,N", [(5, 96), (40, 99), (200, 264), (200, 265)])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("types", ["--f", "ffb", "bbf", "f-b", "-bb", "bff"])
def test_linear_epilogues(M, N, kind, types):
    """bias, residual and output types, with and without each; the residual has a row stride."""
    t = {"f": torch.float32, "b": torch.bfloat16}
    ops = linear_case(M + N, M, N, 256)
    bias = None if types[0] == "-" else rand(1, N, dtype=t[types[0]])
    residual = None if types[1] == "-" else rand(2, M, N + 3, dtype=t[types[1]])[:, 2:2 + N]
    y = fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=act_code(kind), residual=residual, out_dtype=t[types[2]])
    assert y.dtype == t[types[2]]
    check_linear(ops, y, kind, bias, residual)


@pytest.mark.parametrize("M,N,types", [(300, 576, "fff"), (300, 580, "bbf"), (257, 333, "bfb"), (64, 1160, "ffb")])
@pytest.mark.parametrize("kind", ["gelu", "relu"])
@pytest.mark.parametrize("tile", ["128x128", "256x192", "256x256", "256x288"])
@pytest.mark.parametrize("pow2", [False, True])
def test_linear_epilogue_on_every_tile(M, N, types, kind, tile, pow2, monkeypatch):
    monkeypatch.setenv("FG_GEMM_TILE", tile)
    t = {"f": torch.float32, "b": torch.bfloat16}
    ops = linear_case(M + N, M, N, 384, pow2)
    bias, residual = rand(1, N, dtype=t[types[0]]), rand(2, M, N, dtype=t[types[1]])
    y = torch.full((M, N), float("nan"), dtype=t[types[2]], device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=act_code(kind), residual=residual, y=y, pow2=pow2)
    check_linear(ops, y, kind, bias, residual)


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (128, 128, 256), (129, 257, 384), (640, 4096, 1024), (1000, 3001, 512),
                                   (300, 200, 640), (130, 130, 768), (5, 2056, 1152), (256, 128, 4736), (2048, 2056, 256), (1000, 3000, 512),
                                   (1, 1, 5120), (300, 200, 5248), (64, 130, 5376), (129, 264, 5504)])
@pytest.mark.parametrize("pow2", [False, True])
def test_linear_on_small_tiles(M, N, K, pow2, monkeypatch):
    """The 128x128 tiles with two stages and, from 40 blocks of 128 on, with four."""
    monkeypatch.setenv("FG_GEMM_TILE", "128x128")
    ops = linear_case(M, M, N, K, pow2)
    bias, residual = rand(1, N), rand(2, M, N)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_SILU, residual=residual, y=y, pow2=pow2)
    check_linear(ops, y, "silu", bias, residual)


@pytest.mark.parametrize("M,K", [(16, 640), (200, 1152), (16, 5120), (200, 5248)])
def test_linear_small_tiles_exact(M, K, monkeypatch):
    """Small whole numbers: the sum is exact, so each output names the stages it was made of."""
    monkeypatch.setenv("FG_GEMM_TILE", "128x128")
    g = torch.Generator().manual_seed(M)
    x, w = torch.randint(-4, 5, (M, K), generator=g).float(), torch.randint(-2, 3, (272, K), generator=g).float()
    sx = torch.exp2(torch.randint(-1, 2, (K // 128, M), generator=g).float())
    sw = torch.exp2(torch.randint(-1, 2, (3, K // 128), generator=g).float())
    want = (x * sx.t().repeat_interleave(128, 1)) @ (w * sw.repeat_interleave(128, 0)[:272].repeat_interleave(128, 1)).t()
    y = fg.fg_fp8_gemm_fprop_epilogue(x.to(torch.float8_e4m3fn).view(torch.uint8).to(device()), sx.to(device()),
                                      w.to(torch.float8_e4m3fn).view(torch.uint8).to(device()), sw.to(device()), out_dtype=torch.float32)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,N,K", [(1, 300, 4224), (16, 77, 8192), (40, 300, 4224), (10, 4100, 384), (30, 3001, 256), (17, 4100, 640),
                                   (32, 4097, 256), (100, 1030, 640), (333, 515, 1280), (300, 1400, 256), (1000, 1000, 256),
                                   (999, 1013, 384), (1500, 1024, 256), (1490, 1013, 384), (1985, 770, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_streaming_shapes(M, N, K, dtype):
    """Every workgroup shape of the kernel that streams the weights, whole and ragged, short and long contractions."""
    ops = linear_case(M, M, N, K)
    bias, residual = rand(1, N), rand(2, M, N + 1, dtype=dtype)[:, 1:]
    y = torch.full((M, N), float("nan"), dtype=dtype, device=device())
    fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_GELU_TANH, residual=residual, y=y)
    check_linear(ops, y, "gelu", bias, residual)


@pytest.mark.parametrize("M", [1, 16, 64, 65, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_residual_in_place(M, dtype):
    ops = linear_case(M, M, 256, 512)
    r = rand(3, M, 256, dtype=dtype)
    y = r.clone()
    fg.fg_fp8_gemm_fprop_epilogue(*ops, residual=y, y=y, act=fg.FG_ACT_RELU)
    check_linear(ops, y, "relu", None, r)
    assert torch.equal(y, fg.fg_fp8_gemm_fprop_epilogue(*ops, residual=r, out_dtype=dtype, act=fg.FG_ACT_RELU))


@pytest.mark.parametrize("M", [4, 200])
def test_linear_empty_contraction(M):
    ops = linear_case(1, M, 50, 0)
    bias, residual = rand(1, 50), rand(2, M, 50)
    y = fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=fg.FG_ACT_GELU_TANH, residual=residual, out_dtype=torch.float32)
    check_linear(ops, y, "gelu", bias, residual)


@pytest.mark.parametrize("M,N", [(100, 384), (300, 520), (512, 1024), (257, 777)])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("tile", ["256x192", "256x256", "256x288"])
def test_linear_without_epilogue_is_the_fprop(M, N, pow2, tile, monkeypatch):
    """On the GEMM tiles the sums are the Fprop's own, bit for bit."""
    monkeypatch.setenv("FG_GEMM_TILE", tile)
    ops = linear_case(9, M, N, 512, pow2)
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(fg.fg_fp8_gemm_fprop_epilogue(*ops, out_dtype=dtype, pow2=pow2),
                           fg.fg_fp8_gemm_fprop(*ops, out_dtype=dtype, pow2=pow2))


@pytest.mark.parametrize("M", [1, 5, 16, 31, 64])
def test_linear_few_rows_exact(M):
    """Small whole numbers and scales of 1: every order of summation gives the exact sum."""
    K, N = 1152, 272
    g = torch.Generator().manual_seed(M)
    x = torch.randint(-4, 5, (M, K), generator=g).float()
    w = torch.randint(-2, 3, (N, K), generator=g).float()
    ops = (x.to(torch.float8_e4m3fn).view(torch.uint8).to(device()), torch.ones(K // 128, M, device=device()),
           w.to(torch.float8_e4m3fn).view(torch.uint8).to(device()), torch.ones((N + 127) // 128, K // 128, device=device()))
    y = fg.fg_fp8_gemm_fprop_epilogue(*ops, out_dtype=torch.float32)
    assert torch.equal(y.cpu(), x @ w.t())


# ---- activation and checkpoint ----------------------------------------------------------------------------

def wide_values(seed, rows, W, dtype=torch.bfloat16):
    """Columns of different magnitudes, a row and a tile of zeros, values far beyond the activations' bends."""
    z = rand(seed, rows, W, dtype=torch.float32)
    z = z * torch.logspace(-3, 1.5, W, device=z.device)[torch.randperm(W, generator=torch.Generator().manual_seed(seed)).to(z.device)]
    if rows > 2:
        z[1] = 0
        z[2, :128] = 0
    return z.to(dtype)


@pytest.mark.parametrize("rows,F", [(1, 128), (7, 256), (16, 128), (33, 384), (130, 640), (256, 1024)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("pow2", [False, True])
def test_act_forward(rows, F, gated, kind, pow2):
    W = F * (1 + gated)
    z = torch.full((rows, W + 8), float("nan"), dtype=torch.bfloat16, device=device())[:, :W]     # a row stride
    z.copy_(wide_values(rows + F, rows, W))
    zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, act_code(kind), gated=gated, pow2=pow2)
    q, s = fg.fg_quantize_act_1x128(z, pow2=pow2)
    assert torch.equal(zq, q) and torch.equal(sz, s)
    z64 = z.double()
    a, err = ref.act(z64[:, :F], kind)[0], ref.grad_error(z64[:, :F], kind) * z64[:, :F].abs().clamp(max=1)
    if kind in ("none", "relu"):
        err = torch.zeros_like(a)
    if gated:
        err = err * z64[:, F:].abs() + ref.EPS24 * (a * z64[:, F:]).abs()
        a = a * z64[:, F:]
    ref.check_tiles(aq, sa, a, err, pow2, "a")


def test_act_forward_of_every_finite_value():
    """Every finite bf16 value through each activation: nothing but finite values, signs and limits kept."""
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = bits[torch.isfinite(bits)]
    z = torch.cat([z, z.new_zeros(-len(z) % 128)]).view(-1, 128)[:, torch.randperm(128, generator=torch.Generator().manual_seed(1))]
    # one magnitude to a tile, so that each tile's values survive their scale
    z = z[:, :].contiguous().to(device())
    for kind in ("relu", "gelu", "silu"):
        zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, act_code(kind))
        z64 = z.double()
        a = ref.act(z64, kind)[0]
        a = torch.where(torch.isnan(a), torch.relu(z64), a)        # z^3 beyond float64 never happens; inf * 0 would
        assert bool(torch.isfinite(sa).all())
        ref.check_tiles(aq, sa, a, (1e-6 + 4 * ref.grad_error(z64.clamp(-100, 100), kind)) * z64.abs().clamp(max=1) + 2 * ref.EPS24 * a.abs(),
                        False, kind)
        r = fg.fg_act_checkpoint_bwd(zq, sz, torch.ones(z.shape, device=device()), act_code(kind), token_tiles=False,
                                     recompute=False)
        slope = ref.rows_values(r.dzq_cols, r.sdz_cols)
        assert bool(torch.isfinite(slope).all()) and float(slope.min()) > -0.2 and float(slope.max()) < 1.25


def bwd_reference(zq, sz, da, kind, gated):
    z, F, d = ref.rows_values(zq, sz), da.shape[1], da.double()
    a, slope = ref.act(z[:, :F], kind)
    ge = ref.grad_error(z[:, :F], kind)
    if not gated:
        return d * slope, d.abs() * (ge + ref.EPS24), a, ge * z.abs().clamp(max=1) + 2 * ref.EPS24 * a.abs()
    up = z[:, F:]
    dz = torch.cat([d * up * slope, d * a], 1)
    ae = ge * z[:, :F].abs().clamp(max=1) + 2 * ref.EPS24 * a.abs()
    err = torch.cat([(d * up).abs() * (ge + 4 * ref.EPS24), d.abs() * (ae + 2 * ref.EPS24 * a.abs())], 1)
    return dz, err, a * up, ae * up.abs() + 4 * ref.EPS24 * (a * up).abs()


@pytest.mark.parametrize("rows,F", [(128, 128), (256, 384), (640, 256)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("da_type,pow2", [(torch.float32, False), (torch.bfloat16, False), (torch.float32, True)])
def test_act_backward(rows, F, gated, kind, da_type, pow2):
    W = F * (1 + gated)
    zq, sz = fg.fg_quantize_act_1x128(wide_values(rows + F, rows, W))
    da = wide_values(rows, rows, F + 8, torch.float32).mul(1e-3).to(da_type)[:, :F]
    r = fg.fg_act_checkpoint_bwd(zq, sz, da, act_code(kind), gated=gated, pow2=pow2, bias_grad=True)
    dz, err, a, aerr = bwd_reference(zq, sz, da, kind, gated)
    ref.check_tiles(r.dzq_cols, r.sdz_cols, dz, err, pow2, "dz along the columns")
    ref.check_tiles(r.dzq_rows, r.sdz_rows, dz.t().contiguous(), err.t().contiguous(), pow2, "dz along the rows")
    ref.check_tiles(r.aq_rows, r.sa_rows, a.t().contiguous(), aerr.t().contiguous(), pow2, "a along the rows")
    # at most 12 additions deep inside a row block, then one for each block
    tol = err.sum(0) + (12 + rows / 128) * ref.EPS24 * dz.abs().sum(0)
    assert bool(((r.dbias.double() - dz.sum(0)).abs() <= tol).all())


@pytest.mark.parametrize("rows", [1, 5, 127, 129, 300])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_act_backward_ragged_rows(rows, gated, bias):
    """Any number of rows without tilings along them; memory behind the last row stays as it was."""
    F = 256
    W = F * (1 + gated)
    zq, sz = fg.fg_quantize_act_1x128(wide_values(rows, rows, W))
    da = rand(rows, rows, F, dtype=torch.float32)
    guard = torch.full((rows + 3, W), 0x55, dtype=torch.uint8, device=device())
    scales = torch.full(((W // 128) * rows + 64,), 7.0, device=device())
    out = fg.ActGrad(guard[:rows], scales[:(W // 128) * rows].view(W // 128, rows), None, None, None, None, None)
    r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_SILU, gated=gated, token_tiles=False, recompute=False,
                                 bias_grad=bias, out=out)
    assert r.dzq_rows is None and r.aq_rows is None and (r.dbias is not None) == bias
    assert bool((guard[rows:] == 0x55).all()) and bool((scales[(W // 128) * rows:] == 7.0).all())
    dz, err, _, _ = bwd_reference(zq, sz, da, "silu", gated)
    ref.check_tiles(r.dzq_cols, r.sdz_cols, dz, err, False, "dz")
    if bias:
        tol = err.sum(0) + (12 + rows / 128) * ref.EPS24 * dz.abs().sum(0)
        assert bool(((r.dbias.double() - dz.sum(0)).abs() <= tol).all())


@pytest.mark.parametrize("token_tiles,recompute,bias", [(True, False, False), (False, True, False), (False, True, True),
                                                        (True, False, True), (False, False, True)])
def test_act_backward_parts(token_tiles, recompute, bias):
    """Each optional output is the same alone as with the others."""
    zq, sz = fg.fg_quantize_act_1x128(wide_values(3, 256, 512))
    da = rand(4, 256, 256, dtype=torch.float32)
    every = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_GELU_TANH, gated=True, bias_grad=True)
    r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_GELU_TANH, gated=True, token_tiles=token_tiles,
                                 recompute=recompute, bias_grad=bias)
    for a, b in zip(r, every):
        assert a is None or torch.equal(a, b)


def test_act_backward_identity_is_the_quantizer():
    """act NONE and RELU hand bf16 gradients through unrounded: their codes are the quantizers' own, bit for bit."""
    da = wide_values(1, 256, 384)
    zq, sz = fg.fg_quantize_act_1x128(wide_values(2, 256, 384))
    for pow2 in (False, True):
        want = fg.fg_quantize_act_1x128_both(da, pow2=pow2)
        r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_NONE, pow2=pow2, recompute=False)
        for a, b in zip(r[:4], want):
            assert torch.equal(a, b)
        r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_RELU, pow2=pow2, recompute=False)
        on = (ref.rows_values(zq, sz) > 0).to(torch.bfloat16)
        for a, b in zip(r[:4], fg.fg_quantize_act_1x128_both(da * on, pow2=pow2)):
            assert torch.equal(a.where(a != 0x80, 0) if a.dtype == torch.uint8 else a,
                               b.where(b != 0x80, 0) if b.dtype == torch.uint8 else b)     # signs of zeros apart


@pytest.mark.parametrize("exponent", [-126, -120, -100, -90, -60, 60, 100])
def test_act_scales_of_every_size(exponent):
    """Tiles whose scales lie far from 1, down to the smallest normal one."""
    z = (rand(1, 128, 256, dtype=torch.float32) * 2.0 ** exponent).to(torch.bfloat16)
    zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_RELU)
    ref.check_tiles(aq, sa, torch.relu(z.double()), torch.zeros_like(z.double()), False, "a")
    r = fg.fg_act_checkpoint_bwd(zq, sz, z, fg.FG_ACT_NONE, recompute=False)
    for a, b in zip(r[:4], fg.fg_quantize_act_1x128_both(z)):
        assert torch.equal(a, b)


def test_act_gradient_against_differences():
    """The gradient of sum(da * act(z^)) from the checkpoint, against central differences of the forward in 64 bits."""
    zq, sz = fg.fg_quantize_act_1x128(rand(1, 128, 256, std=2.0))
    da = rand(2, 128, 128, dtype=torch.float32)
    h = 1e-5
    for kind in ("gelu", "silu"):
        r = fg.fg_act_checkpoint_bwd(zq, sz, da, act_code(kind), gated=True, recompute=False)
        z = ref.rows_values(zq, sz)
        gate, up = z[:, :128], z[:, 128:]
        dgate = da.double() * up * (ref.act(gate + h, kind)[0] - ref.act(gate - h, kind)[0]) / (2 * h)
        dup = da.double() * ref.act(gate, kind)[0] * ((up + h) - (up - h)) / (2 * h)
        dz = torch.cat([dgate, dup], 1)
        # differences: h^2 / 6 |act'''| < 1e-10, and 1e-16 |act| / h < 1e-10
        _, err, _, _ = bwd_reference(zq, sz, da, kind, True)
        ref.check_tiles(r.dzq_cols, r.sdz_cols, dz, err + 1e-9 * (1 + da.double().abs().repeat(1, 2)) * (1 + z.abs()), False, kind)


@pytest.mark.parametrize("pow2", [False, True])
def test_act_overflow_stays_visible(pow2):
    """A product that overflows becomes a NaN code under a finite scale; the other tiles are what they are without it."""
    z = rand(1, 128, 512)
    z[3, 10], z[3, 266] = 3e38, 3e38
    zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_SILU, gated=True, pow2=pow2)
    assert bool(torch.isfinite(sa).all()) and bool(torch.isfinite(sz).all()) and not bool(((zq & 0x7F) == 0x7F).any())
    assert ((aq & 0x7F) == 0x7F).nonzero().tolist() == [[3, 10]]
    z = rand(2, 128, 512) + 4
    z[5, 140] = z[5, 396] = 4
    zq, sz = fg.fg_quantize_act_1x128(z)
    da = torch.ones(128, 256, device=device())
    calm = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_SILU, gated=True, pow2=pow2)
    da[5, 140] = 3.4e38
    r = fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_SILU, gated=True, pow2=pow2, bias_grad=True)
    for s in (r.sdz_cols, r.sdz_rows, r.sa_rows):
        assert bool(torch.isfinite(s).all()) and bool((s > 0).all())
    assert ((r.dzq_cols & 0x7F) == 0x7F).nonzero().tolist() == [[5, 140], [5, 396]]
    assert ((r.dzq_rows & 0x7F) == 0x7F).nonzero().tolist() == [[140, 5], [396, 5]]
    keep = torch.ones(128, dtype=torch.bool)
    keep[5] = False
    assert torch.equal(r.dzq_cols[keep.to(device())], calm.dzq_cols[keep.to(device())]) and torch.equal(r.aq_rows, calm.aq_rows)
    assert (~torch.isfinite(r.dbias)).nonzero().flatten().tolist() == [140, 396]


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_linear_nan_stays_visible(M, kind):
    ops = linear_case(M, M, 136, 256, False)
    bias = rand(1, 136)
    bias[7] = float("nan")
    y = fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=bias, act=act_code(kind))
    assert bool(torch.isnan(y[:, 7]).all()) and int(torch.isnan(y).sum()) == M


def test_act_empty():
    dev = device()
    z = torch.empty((0, 256), dtype=torch.bfloat16, device=dev)
    zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_SILU, gated=True)
    assert zq.shape == (0, 256) and aq.shape == (0, 128)
    r = fg.fg_act_checkpoint_bwd(zq, sz, torch.empty((0, 128), device=dev), fg.FG_ACT_SILU, gated=True, bias_grad=True)
    assert torch.equal(r.dbias, torch.zeros(256, device=dev))       # the sums of no rows


# ---- mixture of experts ---------------------------------------------------------------------------------

def experts(seed, E, H, I):
    w1, w2 = rand(seed, E * 2 * I, H, std=H ** -0.5), rand(seed + 1, E * H, I, std=I ** -0.5)
    q1, s1 = fg.fg_quantize_w_128x128(w1)
    q2, s2 = fg.fg_quantize_w_128x128(w2)
    return (q1.view(E, 2 * I, H), s1.view(E, 2 * I // 128, H // 128), q2.view(E, H, I), s2.view(E, H // 128, I // 128))


def routing(seed, T, topk, total, E):
    g = torch.Generator().manual_seed(seed)
    score, ids = torch.rand(T, total, generator=g).topk(topk, dim=1)
    ids = torch.where(ids < E, ids, -1)
    return ids.to(torch.int32).to(device()), score.softmax(1).to(device())


def check_moe(y, args, kind, pow2):
    want, bound = ref.moe(*args, kind, pow2)
    assert bool(torch.isfinite(y).all())
    bound = bound + 2.0 ** -20 * want.abs()
    if y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    far = (y.double() - want).abs() - bound
    assert float(far.max()) <= 0, float(far.max())
    # the bound above is a worst case over all hidden values next to a border; their signs differ, so the whole is
    # far closer: within three times the two roundings to 8 bits of the hidden values that the bound is made of
    norm = float(want.norm())
    if norm > 0:
        assert float((y.double() - want).norm()) <= 2.0 ** -6 * norm


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("E,total,topk", [(1, 1, 1), (8, 8, 2), (8, 8, 8), (5, 40, 4), (64, 64, 6)])
@pytest.mark.parametrize("H,I,kind,pow2", [(256, 128, "silu", False), (384, 640, "gelu", True)])
def test_moe(T, E, total, topk, H, I, kind, pow2):
    w = experts(E + H, E, H, I)
    x = rand(T, T, H)
    ids, weights = routing(T + E, T, topk, total, E)
    y = fg.fg_moe_few_tokens(x, ids, weights, *w, act=act_code(kind), pow2=pow2)
    check_moe(y, (x, ids, weights, *w), kind, pow2)
    nobody = (ids < 0).all(1)
    assert bool((y[nobody] == 0).all())


@pytest.mark.parametrize("T", [3, 20, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_moe_odd_routing(T, dtype):
    """Ids out of range with NaN weights, tokens that nobody takes with NaN inputs, an expert chosen twice, an expert
    that everybody chose, and a strided x and y."""
    E, H, I, topk = 6, 256, 256, 4
    w = experts(1, E, H, I)
    x = torch.zeros(T, H + 8, dtype=torch.bfloat16, device=device())[:, :H]
    x.copy_(rand(2, T, H))
    ids, weights = routing(3, T, topk, E, E)
    ids[:, 0] = 2
    ids[1] = torch.tensor([4, 4, -7, 4], dtype=torch.int32)
    ids[2] = torch.tensor([E, 1 << 30, -1, -(1 << 31)], dtype=torch.int32)
    weights[1, 2] = float("nan")
    weights[2] = float("nan")
    x[2] = float("nan")
    y = torch.full((T, H + 5), 9.0, dtype=dtype, device=device())
    fg.fg_moe_few_tokens(x, ids, weights, *w, act=fg.FG_ACT_SILU, y=y[:, :H])
    assert bool((y[:, H:] == 9.0).all()) and bool((y[2, :H] == 0).all())
    x, weights = x.clone(), weights.clone()
    x[2] = 0
    weights[1, 2] = weights[2] = 0
    check_moe(y[:, :H], (x, ids, weights, *w), "silu", False)


@pytest.mark.parametrize("T", [1, 7, 16, 18, 64])
def test_moe_exact(T):
    """Weights with one entry a row and powers of two everywhere: every product and sum is exact, so each output
    names the elements it was made of."""
    E, H, I, topk = 9, 384, 256, 3
    g = torch.Generator().manual_seed(T)
    x = torch.exp2(torch.randint(-2, 3, (T, H), generator=g).float()) * (1 - 2 * torch.randint(0, 2, (T, H), generator=g))
    w1, w2 = torch.zeros(E, 2 * I, H), torch.zeros(E, H, I)
    pick1, pick2 = torch.randint(0, H, (E, 2 * I, 1), generator=g), torch.randint(0, I, (E, H, 1), generator=g)
    w1.scatter_(2, pick1, torch.exp2(torch.randint(-1, 2, (E, 2 * I, 1), generator=g).float()))
    w2.scatter_(2, pick2, torch.exp2(torch.randint(-1, 2, (E, H, 1), generator=g).float()))
    ids = torch.rand(T, E + 3, generator=g).topk(topk, dim=1).indices.to(torch.int32)      # some beyond E
    weights = torch.exp2(torch.randint(-3, 1, (T, topk), generator=g).float())
    codes = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8).to(device())  # noqa: E731
    y = fg.fg_moe_few_tokens(x.to(torch.bfloat16).to(device()), ids.to(device()), weights.to(device()), codes(w1),
                             torch.ones(E, 2 * I // 128, H // 128, device=device()), codes(w2),
                             torch.ones(E, H // 128, I // 128, device=device()), act=fg.FG_ACT_NONE, out_dtype=torch.float32,
                             pow2=True)
    want = torch.zeros(T, H)
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            if e < E:
                gu = w1[e] @ x[t]
                want[t] += weights[t, j] * (w2[e] @ (gu[:I] * gu[I:]))
    assert torch.equal(y.cpu(), want)


def test_moe_is_the_training_layer():
    """The layer for a few tokens against the training operators on the same weights: quantize, grouped Fprop, gated
    activation with its checkpoint, grouped Fprop, weighted sum."""
    T, E, H, I, topk = 24, 4, 512, 256, 2
    q1, s1, q2, s2 = experts(5, E, H, I)
    x = rand(6, T, H)
    ids, weights = routing(7, T, topk, E, E)
    order = ids.flatten().long().argsort(stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=device())
    offsets[1:] = torch.bincount(ids.flatten().long(), minlength=E).cumsum(0)
    xq, sx = fg.fg_quantize_act_1x128(x[order // topk].contiguous())
    z = fg.fg_fp8_grouped_gemm(xq, sx, q1, s1, offsets)
    _, _, aq, sa = fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_SILU, gated=True)
    out = fg.fg_fp8_grouped_gemm(aq, sa, q2, s2, offsets, out_dtype=torch.float32)
    want = torch.zeros(T, H, dtype=torch.float64, device=device())
    want.index_add_(0, order // topk, out.double() * weights.flatten()[order, None].double())
    y = fg.fg_moe_few_tokens(x, ids, weights, q1, s1, q2, s2, out_dtype=torch.float32)
    # z was rounded to bf16 there (2^-8 of each factor) and the hidden values to 8 bits in both (2^-4, where the two
    # differ): independent errors of many terms, so within 2^-5 of the whole
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -5


@pytest.mark.parametrize("T,E,topk,H,I", [(9, 48, 6, 1024, 512), (48, 32, 6, 512, 1024), (64, 40, 8, 2048, 256), (16, 16, 16, 384, 1152)])
def test_moe_split_down_projection(T, E, topk, H, I):
    """Narrow models with many experts: the down-projection's column blocks are shared between workgroups."""
    w = experts(E, E, H, I)
    x = rand(T, T, H)
    ids, weights = routing(T + E, T, topk, E, E)
    for dtype in (torch.float32, torch.bfloat16):
        y = fg.fg_moe_few_tokens(x, ids, weights, *w, out_dtype=dtype)
        check_moe(y, (x, ids, weights, *w), "silu", False)


def test_moe_every_tile_count():
    """Experts with 0, 1, 15, 16, 17, 32, 33, 48, 49 and 64 tokens in one call."""
    counts = [0, 1, 15, 16, 17, 32, 33, 48, 49, 64]
    T, E, H, I = 64, len(counts), 256, 256
    ids = torch.full((T, E), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    for e, n in enumerate(counts):
        ids[torch.randperm(T, generator=g)[:n], e] = e
    ids = ids[:, torch.randperm(E, generator=g)].to(device())
    weights = torch.rand(T, E, generator=g).to(device())
    w = experts(3, E, H, I)
    x = rand(4, T, H)
    check_moe(fg.fg_moe_few_tokens(x, ids, weights, *w, out_dtype=torch.float32), (x, ids, weights, *w), "silu", False)


def test_moe_empty():
    w = experts(1, 2, 256, 128)
    dev = device()
    y = fg.fg_moe_few_tokens(torch.empty((0, 256), dtype=torch.bfloat16, device=dev), torch.empty((0, 2), dtype=torch.int32, device=dev),
                             torch.empty((0, 2), device=dev), *w)
    assert y.shape == (0, 256)
    # no hidden values: sums of nothing
    y = fg.fg_moe_few_tokens(rand(1, 3, 256), torch.zeros((3, 1), dtype=torch.int32, device=dev), torch.ones((3, 1), device=dev),
                             w[0][:, :0].contiguous(), w[1][:, :0].contiguous(), w[2][:, :, :0].contiguous(), w[3][:, :, :0].contiguous())
    assert bool((y == 0).all())


def test_moe_most_choices():
    """64 tokens with 32 choices each among 2048 experts: the largest lists the layer keeps on chip."""
    E, H, I = 2048, 128, 128
    q1, s1, q2, s2 = experts(1, 8, H, I)
    big = [t.repeat(E // 8, *(1,) * (t.dim() - 1)) for t in (q1, s1, q2, s2)]
    ids, weights = routing(2, 64, 32, E, E)
    x = rand(3, 64, H)
    y = fg.fg_moe_few_tokens(x, ids, weights, *big, out_dtype=torch.float32)
    check_moe(y, (x, ids % 8, weights, q1, s1, q2, s2), "silu", False)


@pytest.mark.parametrize("T,topk", [(1, 32), (2, 32), (3, 32), (16, 4), (16, 32), (13, 5), (17, 32)])
def test_moe_choices_again_and_out_of_range(T, topk):
    """Up to 32 choices a token that repeat and miss the experts, on both sides of 64 choices and of 16 tokens."""
    E, H, I = 12, 256, 128
    w = experts(1, E, H, I)
    g = torch.Generator().manual_seed(T * topk)
    ids = torch.randint(-2, E + 2, (T, topk), generator=g, dtype=torch.int32).to(device())
    weights = (torch.rand(T, topk, generator=g) / topk).to(device())
    x = rand(2, T, H)
    y = fg.fg_moe_few_tokens(x, ids, weights, *w, out_dtype=torch.float32)
    check_moe(y, (x, ids, weights, *w), "silu", False)


# ---- together -------------------------------------------------------------------------------------------

def mlp_step(x, dy, w1, b1, w2, b2, gated, kind):
    """A feed-forward block in training: y = act(x W1^T + b1) W2^T + b2 + x, and its gradients."""
    xq, sx, xtq, sxt, w1q, s1 = fg.fg_quantize_fprop_operands(x, w1)
    w2q, s2 = fg.fg_quantize_w_128x128(w2)
    z = fg.fg_fp8_gemm_fprop_epilogue(xq, sx, w1q, s1, bias=b1)
    zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(z, act_code(kind), gated=gated)
    y = fg.fg_fp8_gemm_fprop_epilogue(aq, sa, w2q, s2, bias=b2, residual=x)
    dyq, sdy, dytq, sdyt = fg.fg_quantize_act_1x128_both(dy)
    da = fg.fg_fp8_gemm_dgrad(dyq, sdy, w2q, s2)
    g = fg.fg_act_checkpoint_bwd(zq, sz, da, act_code(kind), gated=gated, bias_grad=True)
    dw2 = fg.fg_fp8_gemm_wgrad(dytq, sdyt, g.aq_rows, g.sa_rows)
    dx = fg.fg_fp8_gemm_dgrad(g.dzq_cols, g.sdz_cols, w1q, s1)
    dw1 = fg.fg_fp8_gemm_wgrad(g.dzq_rows, g.sdz_rows, xtq, sxt)
    return y, dx, dw1, g.dbias, dw2


@pytest.mark.parametrize("gated,kind", [(True, "silu"), (False, "gelu")])
def test_block_in_training(gated, kind):
    """Outputs and gradients of the whole block against autograd in 64 bits on the unquantized values. Every factor
    is rounded to 4 significant bits (2^-4 at most, 2^-5.8 root mean square) at most four times on the way to an
    output, with independent signs: within 2^-3 of the whole."""
    M, H, F = 256, 384, 512
    W = F * (1 + gated)
    x, dy = rand(1, M, H), rand(2, M, H, std=1e-2)
    w1, w2 = rand(3, W, H, std=H ** -0.5), rand(4, H, F, std=F ** -0.5)
    b1, b2 = rand(5, W, std=0.3, dtype=torch.float32), rand(6, H, std=0.3)
    got = mlp_step(x, dy, w1, b1, w2, b2, gated, kind)
    v = [t.double().requires_grad_() for t in (x, w1, b1, w2)]
    z = v[0] @ v[1].t() + v[2]
    a = ref.act(z[:, :F], kind)[0] * (z[:, F:] if gated else 1)
    y = a @ v[3].t() + b2.double() + x.double()
    dx, dw1, db1, dw2 = torch.autograd.grad(y, v, dy.double())
    for name, a, b in zip(("y", "dx", "dw1", "db1", "dw2"), got, (y, dx, dw1, db1, dw2)):
        assert float((a.double() - b.detach()).norm() / b.detach().norm()) <= 2.0 ** -3, name


def test_block_in_a_graph():
    """The block's forward, backward and the layer for a few tokens captured once and replayed on new inputs."""
    M, H, F = 128, 256, 256
    w1, w2 = rand(3, 2 * F, H, std=H ** -0.5), rand(4, H, F, std=F ** -0.5)
    b1, b2 = rand(5, 2 * F, dtype=torch.float32), rand(6, H)
    we = experts(7, 4, H, 128)
    x, dy = rand(1, M, H), rand(2, M, H)
    ids, weights = routing(1, 40, 2, 6, 4)

    def step():
        return (*mlp_step(x, dy, w1, b1, w2, b2, True, "silu"), fg.fg_moe_few_tokens(x[:40], ids, weights, *we),
                fg.fg_moe_few_tokens(x[:3], ids[:3], weights[:3], *we))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(rand(10 + k, M, H))
        dy.copy_(rand(20 + k, M, H))
        i, w = routing(30 + k, 40, 2, 6, 4)
        ids.copy_(i)
        weights.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), k


def test_same_results_every_time_and_on_two_streams():
    """No result depends on what runs beside it or on what a workspace held."""
    we = experts(7, 8, 512, 256)
    x = rand(1, 48, 512)
    ids, weights = routing(2, 48, 4, 8, 8)
    zq, sz = fg.fg_quantize_act_1x128(rand(3, 512, 512))
    da = rand(4, 512, 256, dtype=torch.float32)
    ops = linear_case(5, 32, 512, 2048)
    need = fg.lib().fg_moe_few_tokens_workspace(48, 4, 512, 256)

    def every(fill):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=device())
        return (fg.fg_moe_few_tokens(x, ids, weights, *we, workspace=ws), fg.fg_moe_few_tokens(x[:9], ids[:9], weights[:9], *we, workspace=ws),
                *fg.fg_act_checkpoint_bwd(zq, sz, da, fg.FG_ACT_SILU, gated=True, bias_grad=True),
                fg.fg_fp8_gemm_fprop_epilogue(*ops, act=fg.FG_ACT_SILU))

    want = every(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(every(0xFF))
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


# ---- refusals through the binding ---------------------------------------------------------------------------

def test_binding_refuses():
    dev = device()
    ops = linear_case(1, 8, 256, 256)
    bad = pytest.raises(fg.Fp8fgError)
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=rand(1, 255))
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, bias=rand(1, 256).half())
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, residual=rand(1, 8, 512)[:, ::2])
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, act=9)
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(ops[0], ops[1][:1], *ops[2:])
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, out_dtype=torch.float16)
    y = torch.zeros(8, 256, device=dev)
    with bad:
        fg.fg_fp8_gemm_fprop_epilogue(*ops, residual=y.view(torch.bfloat16)[:, :256], y=y)     # same memory, another type
    with bad:
        fg.fg_act_checkpoint_fwd(rand(1, 4, 256, dtype=torch.float32), fg.FG_ACT_SILU)
    with bad:
        fg.fg_act_checkpoint_fwd(rand(1, 4, 200), fg.FG_ACT_SILU)
    with bad:
        fg.fg_act_checkpoint_fwd(rand(1, 4, 384), fg.FG_ACT_SILU, gated=True)                 # F = 192
    zq, sz = fg.fg_quantize_act_1x128(rand(1, 100, 256))
    with bad:
        fg.fg_act_checkpoint_bwd(zq, sz, rand(1, 100, 256), fg.FG_ACT_SILU)                   # rows % 128 with token tiles
    with bad:
        fg.fg_act_checkpoint_bwd(zq, sz, rand(1, 100, 128), fg.FG_ACT_SILU, token_tiles=False, recompute=False)
    zq, sz = fg.fg_quantize_act_1x128(rand(1, 256, 256))
    with bad:
        fg.fg_act_checkpoint_bwd(zq, sz, rand(1, 256, 256), fg.FG_ACT_SILU, bias_grad=True,
                                 workspace=torch.empty(8, dtype=torch.uint8, device=dev))
    w = experts(1, 2, 256, 128)
    x, (ids, weights) = rand(1, 65, 256), routing(1, 65, 1, 2, 2)
    with bad:
        fg.fg_moe_few_tokens(x, ids, weights, *w)                                             # more than 64 tokens
    with bad:
        fg.fg_moe_few_tokens(x[:4], ids[:4].long(), weights[:4], *w)
    with bad:
        fg.fg_moe_few_tokens(x[:4], ids[:4], weights[:4], *w, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with bad:
        fg.fg_moe_few_tokens(x[:4], ids[:4], weights[:4].cpu(), *w)
    assert fg.lib().fg_last_hip_error() == 0
