"""The operators at the two ends of a Linear's training step on the GPU, against their definitions in 64 bits: the norm with FP8
tiles, its backward pass, and the orthogonalised update."""
import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests import ffn_ref, train_ref as ref
from tests.ffn_ref import EPS24
from tests.gpu_util import device

pytestmark = pytest.mark.gpu
T = {"f": torch.float32, "b": torch.bfloat16}


def rand(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(device())


def strided(t, extra):
    """The same values, rows `extra` elements further apart."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def rows_like(seed, rows, cols, dtype):
    x = rand(seed, rows, cols) * torch.exp(rand(seed + 1, rows, 1, std=0.5)) + 0.3
    x[:, ::37] *= 15
    return x.to(dtype)


# ---- norm ---------------------------------------------------------------------------------------------

def check_norm(r, x, gamma, beta, layer, eps, pow2, what):
    y, err, mean, mean_err, rstd, rel = ref.norm(x.double(), gamma.double(), None if beta is None else beta.double(), layer, eps)
    ffn_ref.check_tiles(r.q_cols, r.s_cols, y, err, pow2, what)
    if r.q_rows is not None:
        ffn_ref.check_tiles(r.q_rows, r.s_rows, y.t().contiguous(), err.t().contiguous(), pow2, what)
    if r.y is not None:
        assert bool(((r.y.double() - y).abs() <= (y.abs() + err) * 2.0 ** -8 + err).all()), what
    if r.rstd is not None:
        assert bool(((r.rstd.double() - rstd).abs() <= (rel + 2 * EPS24) * rstd).all()), what
        if layer:
            assert bool(((r.mean.double() - mean).abs() <= mean_err + EPS24 * mean.abs()).all()), what


def filled(rows, cols, layer, tokens, y=True):
    """Output buffers that hold something else first."""
    def u8(*s):
        return torch.full(s, 0x7F, dtype=torch.uint8, device=device())

    def f32(*s):
        return torch.full(s, float("nan"), device=device())
    return fg.NormTiles(u8(rows, cols), f32(cols // 128, rows), u8(cols, rows) if tokens else None,
                        f32(rows // 128, cols) if tokens else None,
                        torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device=device()) if y else None,
                        f32(rows) if layer else None, f32(rows))


NORM_SHAPES = [(1, 128), (1, 1024), (3, 384), (5, 640), (17, 512), (2, 8192), (33, 7168), (4, 8320), (3, 12288), (3, 12416), (3, 16384), (2, 16512), (3, 18432),
               (700, 256), (1200, 1152), (600, 4224)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_shapes(rows, cols, kind):
    layer = kind == "layer"
    x, gamma, beta = rows_like(rows + cols, rows, cols, torch.bfloat16), 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    out = filled(rows, cols, layer, False)
    r = fg.fg_norm_quantize(x, gamma, beta if layer else None, kind=getattr(fg, "FG_NORM_" + kind.upper()), with_y=True, out=out)
    assert r.q_cols is out.q_cols and r.y is out.y and r.q_rows is None
    check_norm(r, x, gamma, beta if layer else None, layer, 1e-5, False, (rows, cols, kind))


@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 640), (384, 1024), (128, 8320), (1280, 256), (128, 18432), (8448, 256),
                                       (640, 18432)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("pow2", [False, True])
def test_norm_both_tilings(rows, cols, kind, pow2):
    layer = kind == "layer"
    x, gamma, beta = rows_like(rows + cols, rows, cols, torch.float32), 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    r = fg.fg_norm_quantize(x, gamma, beta, kind=fg.FG_NORM_LAYER if layer else fg.FG_NORM_RMS, pow2=pow2, token_tiles=True,
                            out=filled(rows, cols, layer, True, y=False))
    check_norm(r, x, gamma, beta, layer, 1e-5, pow2, (rows, cols, kind))


@pytest.mark.parametrize("types", ["ff", "fb", "bf", "bb"])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("tokens", [False, True])
def test_norm_types(types, beta, kind, tokens):
    rows, cols = 128 if tokens else 37, 768
    x = strided(rows_like(1, rows, cols, T[types[0]]), 24)
    gamma, b = (1 + rand(2, cols, std=0.2)).to(T[types[1]]), rand(3, cols, std=0.3).to(T[types[1]])
    r = fg.fg_norm_quantize(x, gamma, b if beta else None, kind=fg.FG_NORM_LAYER if kind == "layer" else fg.FG_NORM_RMS, eps=1e-3,
                            token_tiles=tokens, with_y=True)
    check_norm(r, x, gamma, b if beta else None, kind == "layer", 1e-3, False, types)
    if not tokens:
        bare = fg.fg_norm_quantize(x, gamma, b if beta else None, kind=fg.FG_NORM_LAYER if kind == "layer" else fg.FG_NORM_RMS,
                                   eps=1e-3, statistics=False)
        assert bare.mean is None and bare.rstd is None and bare.y is None
        assert torch.equal(bare.q_cols, r.q_cols) and torch.equal(bare.s_cols, r.s_cols)


def odd(*shape, dtype=torch.float32, fill=float("nan")):
    """A buffer that begins one element behind an aligned one."""
    n = 1
    for d in shape:
        n *= d
    return torch.full((n + 1,), fill, dtype=dtype, device=device())[1:].view(*shape)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_fp32_buffers_aligned_to_their_elements(kind):
    """Scales, statistics and the weights' gradients need no more than their elements' alignment."""
    rows, cols, layer = 256, 640, kind == "layer"
    k = fg.FG_NORM_LAYER if layer else fg.FG_NORM_RMS
    x, gamma, beta = rows_like(1, rows, cols, torch.bfloat16), 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    want = fg.fg_norm_quantize(x, gamma, beta, kind=k, token_tiles=True, with_y=True)
    out = fg.NormTiles(torch.empty_like(want.q_cols), odd(cols // 128, rows), torch.empty_like(want.q_rows), odd(rows // 128, cols),
                       torch.empty_like(want.y), odd(rows), odd(rows))
    got = fg.fg_norm_quantize(x, gamma, beta, kind=k, token_tiles=True, with_y=True, out=out)
    assert got.s_cols.data_ptr() % 16 == 4
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    dy = rand(4, rows, cols)
    grad = fg.fg_norm_bwd(x, want.mean, want.rstd, gamma, dy, kind=k, bias_grad=True)
    same = fg.fg_norm_bwd(x, got.mean, got.rstd, gamma, dy, kind=k, bias_grad=True, dgamma=odd(cols), dbeta=odd(cols))
    assert all(torch.equal(a, b) for a, b in zip(same, grad))


def test_norm_far_off_centre():
    """A mean a thousand times the deviation: the squares are summed about the mean."""
    x = rand(1, 9, 2048, std=1.0) + 1000.0
    gamma = torch.ones(2048, device=device())
    check_norm(fg.fg_norm_quantize(x, gamma, with_y=True), x, gamma, None, True, 1e-5, False, "off centre")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_special_rows(kind):
    """Rows of zeros, of one value, tiny and huge rows, and rows that hold a NaN or an infinity beside ordinary ones."""
    rows, cols = 128, 512
    x = rows_like(5, rows, cols, torch.float32)
    x[3] = 0
    x[4] = 7.25
    x[5] *= 1e-30
    x[6] *= 1e15
    clean = x.clone()
    x[10, 7], x[11, 300], x[12, 0] = float("nan"), float("inf"), float("-inf")
    gamma, beta = 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    k = fg.FG_NORM_LAYER if kind == "layer" else fg.FG_NORM_RMS
    r, c = (fg.fg_norm_quantize(v, gamma, beta, kind=k, token_tiles=True, with_y=True) for v in (x, clean))
    good = [i for i in range(rows) if i not in (10, 11, 12)]
    assert torch.equal(r.q_cols[good], c.q_cols[good]) and torch.equal(r.s_cols[:, good], c.s_cols[:, good])
    bad = r.q_cols[10:13] & 0x7F
    assert bool((bad == 0x7F).all()) and bool(torch.isnan(r.y[10:13]).all()) and bool(torch.isnan(r.rstd[10:13]).all())
    assert bool(((r.q_rows[:, 10:13] & 0x7F) == 0x7F).all())
    assert bool(torch.isfinite(r.s_cols).all()) and bool(torch.isfinite(r.s_rows).all())
    sub = x[good]
    part = fg.NormTiles(r.q_cols[good], r.s_cols[:, good].contiguous(), None, None, r.y[good], r.mean[good] if kind == "layer" else None,
                        r.rstd[good])
    check_norm(part, sub, gamma, beta, kind == "layer", 1e-5, False, "special rows")


# ---- backward -----------------------------------------------------------------------------------------

def check_grad(r, x, mean, rstd, gamma, dy, dres, layer, what, before=(0.0, 0.0)):
    rows = x.shape[0]
    dx, err, dg, db, dg_abs, db_abs = ref.norm_grad(x.double(), mean.double() if layer else None, rstd.double(), gamma.double(), dy.double(),
                                                    None if dres is None else dres.double(), layer)
    tol = err + EPS24 * (dx.abs() + err)
    if r.dx.dtype == torch.bfloat16:
        tol = tol + (dx.abs() + tol) * 2.0 ** -8
    assert r.dx.dtype in T.values() and bool(((r.dx.double() - dx).abs() <= tol).all()), (what, float(((r.dx.double() - dx).abs() - tol).max()))
    # additions of a column: a thread's rows, a workgroup's groups, and the partial sums
    depth = -(-rows // 256) + 16 + 16 + 16 + 4
    for got, want, mag, was in ((r.dgamma, dg, dg_abs, before[0]), (r.dbeta, db, db_abs, before[1])):
        if got is not None:
            want = want + was
            assert bool(((got.double() - want).abs() <= depth * EPS24 * (mag + abs(was)) + EPS24 * want.abs()).all()), what


def grad_case(rows, cols, layer, x_type=torch.bfloat16, dy_type=torch.float32):
    x, gamma = rows_like(rows + cols, rows, cols, x_type), 1 + rand(2, cols, std=0.2)
    _, _, mean, _, rstd, _ = ref.norm(x.double(), gamma.double(), None, layer, 1e-5)
    return x, mean.float() if layer else None, rstd.float(), gamma, rand(7, rows, cols, std=1e-3).to(dy_type)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(3000, 128), (2100, 2048), (511, 1024), (512, 2176), (513, 8192), (530, 12288), (520, 16512)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_shapes(rows, cols, kind):
    layer = kind == "layer"
    x, mean, rstd, gamma, dy = grad_case(rows, cols, layer)
    nan = torch.full((cols,), float("nan"), device=device())
    dx = torch.full((rows, cols), float("nan"), device=device())
    ws = torch.full((fg.lib().fg_norm_bwd_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device=device())
    r = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, kind=fg.FG_NORM_LAYER if layer else fg.FG_NORM_RMS, bias_grad=True, dx=dx,
                       dgamma=nan.clone(), dbeta=nan.clone(), workspace=ws)
    assert r.dx is dx
    check_grad(r, x, mean, rstd, gamma, dy, None, layer, (rows, cols, kind))


@pytest.mark.parametrize("types", ["fff-f", "bfbfb", "ffbbf", "bbfbb", "bff-b", "fbbff"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_types(types, kind):
    """x, weight, dy, residual gradient and dx in each type, with strides."""
    layer, rows, cols = kind == "layer", 41, 896
    x, mean, rstd, gamma, dy = grad_case(rows, cols, layer, T[types[0]], T[types[2]])
    gamma = gamma.to(T[types[1]])
    dres = None if types[3] == "-" else strided(rand(9, rows, cols, std=2e-3).to(T[types[3]]), 40)
    r = fg.fg_norm_bwd(strided(x, 8), mean, rstd, gamma, strided(dy, 16), residual_grad=dres, kind=fg.FG_NORM_LAYER if layer else
                       fg.FG_NORM_RMS, out_dtype=T[types[4]], bias_grad=True)
    assert r.dx.dtype == T[types[4]]
    check_grad(r, x, mean, rstd, gamma, dy, dres, layer, types)


@pytest.mark.parametrize("rows,cols", [(300, 1024), (900, 1024), (40, 14336), (530, 14336)])
def test_grad_into_its_residual_and_accumulated(rows, cols):
    x, mean, rstd, gamma, dy = grad_case(rows, cols, True)
    for dtype in T.values():
        dres = rand(9, rows, cols, std=2e-3).to(dtype)
        want = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=dres, out_dtype=dtype, bias_grad=True)
        dx = dres.clone()
        r = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=dx, dx=dx, weight_grad=False)
        assert torch.equal(dx, want.dx) and r.dgamma is None and r.dbeta is None
    twice = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, bias_grad=True, accumulate=True, dgamma=torch.full((cols,), 3.0, device=device()),
                           dbeta=torch.full((cols,), -2.0, device=device()))
    check_grad(twice, x, mean, rstd, gamma, dy, None, True, "accumulate", before=(3.0, -2.0))


@pytest.mark.parametrize("rows,cols", [(70, 384), (40, 5120), (9, 9216), (9, 14336), (512, 128), (513, 128), (600, 640), (520, 5120), (515, 9216), (513, 14336)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_of_either_weight(rows, cols, kind):
    """dgamma or dbeta alone, and neither: the same numbers as together, whatever way the sums are held and joined."""
    layer = kind == "layer"
    x, mean, rstd, gamma, dy = grad_case(rows, cols, layer)
    args = dict(kind=fg.FG_NORM_LAYER if layer else fg.FG_NORM_RMS)
    both = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, bias_grad=True, **args)
    check_grad(both, x, mean, rstd, gamma, dy, None, layer, (rows, cols, kind))
    for weight, bias in ((True, False), (False, True), (False, False)):
        r = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, weight_grad=weight, bias_grad=bias, **args)
        assert torch.equal(r.dx, both.dx) and (r.dgamma is None) != weight and (r.dbeta is None) != bias
        assert not weight or torch.equal(r.dgamma, both.dgamma)
        assert not bias or torch.equal(r.dbeta, both.dbeta)


def test_grad_of_no_rows():
    e = torch.empty(0, 256, device=device())
    v, nan = torch.empty(0, device=device()), torch.full((256,), float("nan"), device=device())
    gamma = torch.ones(256, device=device())
    r = fg.fg_norm_bwd(e, v, v, gamma, e, bias_grad=True, dgamma=nan.clone(), dbeta=nan.clone())
    assert not r.dgamma.any() and not r.dbeta.any() and r.dx.shape == (0, 256)
    kept = torch.full((256,), 5.0, device=device())
    fg.fg_norm_bwd(e, v, v, gamma, e, accumulate=True, dgamma=kept)
    assert bool((kept == 5).all())
    assert fg.fg_norm_quantize(e, gamma).q_cols.shape == (0, 256)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_against_differences(kind):
    """The backward pass against differences of the forward formula in 64 bits, of sum(y w) for a fixed w."""
    layer, rows, cols = kind == "layer", 4, 128
    x, gamma, beta, w = rand(1, rows, cols).double(), 1 + rand(2, cols, std=0.2).double(), rand(3, cols).double(), rand(4, rows, cols).double()

    def loss(x, gamma, beta):
        return float((ref.norm(x, gamma, beta, layer, 1e-5)[0] * w).sum())
    _, _, mean, _, rstd, _ = ref.norm(x, gamma, beta, layer, 1e-5)
    r = fg.fg_norm_bwd(x.float(), mean.float() if layer else None, rstd.float(), gamma.float(), w.float(), kind=fg.FG_NORM_LAYER if layer else
                       fg.FG_NORM_RMS, out_dtype=torch.float32, bias_grad=True)
    h = 1e-5
    for i, c in ((0, 0), (1, 17), (3, 127), (2, 64)):
        step = torch.zeros_like(x)
        step[i, c] = h
        # the difference's own error is of the order of h^2 and 1e-16 loss / h; the gradient is fp32
        want = (loss(x + step, gamma, beta) - loss(x - step, gamma, beta)) / (2 * h)
        assert abs(float(r.dx[i, c]) - want) <= 1e-5 * max(1.0, abs(want)), (i, c)
    for c in (0, 31, 127):
        step = torch.zeros_like(gamma)
        step[c] = h
        for got, f in ((r.dgamma, lambda s: loss(x, gamma + s, beta)), (r.dbeta, lambda s: loss(x, gamma, beta + s))):
            want = (f(step) - f(-step)) / (2 * h)
            assert abs(float(got[c]) - want) <= 1e-5 * max(1.0, abs(want)), c


# ---- orthogonalised update ----------------------------------------------------------------------------

def gradient(seed, n, k, dtype=torch.float32, tokens=None):
    t = tokens or 2 * min(n, k) + 16
    return (rand(seed, t, n, std=1e-3).t() @ rand(seed + 1, t, k)).to(dtype)


def dirty_workspace(batch, n, k):
    return torch.full((fg.lib().fg_orthogonalize_workspace(batch, n, k),), 0xFF, dtype=torch.uint8, device=device())


SIDES = [(1, 1), (1, 200), (200, 1), (2, 3), (5, 64), (63, 65), (64, 64), (65, 130), (128, 128), (129, 128), (127, 300), (257, 129),
         (200, 1000), (1000, 333), (256, 1024), (520, 512), (640, 2112)]


@pytest.mark.parametrize("n,k", SIDES)
@pytest.mark.parametrize("dtype", ["f", "b"])
def test_update_sizes(n, k, dtype):
    g = gradient(n + k, n, k, T[dtype])
    out = torch.full((n, k), float("nan"), dtype=torch.bfloat16, device=device())
    r = fg.fg_orthogonalize(g, scale=0.5, out=out, workspace=dirty_workspace(1, n, k))
    assert r is out
    check = ref.orthogonalize(g.double(), scale=0.5)
    ref.check_update(out, *check, (n, k))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_update_steps(steps):
    g = gradient(3, 150, 200)
    ref.check_update(fg.fg_orthogonalize(g, steps=steps), *ref.orthogonalize(g.double(), steps=steps), steps)


def test_update_other_coefficients():
    """The cubic iteration, whose singular values all go to one."""
    g = gradient(3, 96, 160)
    out = fg.fg_orthogonalize(g, steps=30, coefficients=(1.5, -0.5, 0.0))
    ref.check_update(out, *ref.orthogonalize(g.double(), steps=30, coefficients=(1.5, -0.5, 0.0)))
    s = torch.linalg.svdvals(out.double().cpu())
    assert float((s - 1).abs().max()) < 0.02          # fp16 and bf16 roundings of a matrix of norm sqrt(96)


@pytest.mark.parametrize("shape", [(3, 70, 90), (2, 200, 64), (5, 1, 33), (4, 130, 260)])
def test_update_batches_and_strides(shape):
    b, n, k = shape
    g = torch.stack([gradient(i, n, k) for i in range(b)])
    out = fg.fg_orthogonalize(g, workspace=dirty_workspace(*shape))
    for i in range(b):
        ref.check_update(out[i], *ref.orthogonalize(g[i].double()), (shape, i))
    wide = torch.full((b, n, k + 5), float("nan"), device=device())
    wide[..., 3:3 + k] = g
    assert torch.equal(fg.fg_orthogonalize(wide[..., 3:3 + k]), out)
    assert torch.equal(fg.fg_orthogonalize(g[0]), out[0])


@pytest.mark.parametrize("batch,n,k,steps", [(1, 1100, 4200, 2), (1, 2040, 2100, 1), (3, 1030, 2100, 2), (1, 4096, 4160, 1), (8, 2048, 2048, 2), (9, 2050, 1990, 1),
                                               (1, 2048, 8448, 2), (1, 2000, 8400, 2), (8, 2000, 2040, 1), (8, 512, 1024, 2), (8, 1024, 2050, 2),
                                               (1, 2000, 10400, 2), (8, 2048, 7168, 1), (8, 2000, 7000, 1)])
def test_update_on_every_tile(batch, n, k, steps):
    """Sizes whose products take the 128 x 128 tiles in both forms, the 256 x 256 ones, and those with a rest in quarters, whose
    matrices are the last."""
    g = torch.stack([gradient(i, n, k) for i in range(batch)])
    out = fg.fg_orthogonalize(g, steps=steps, out=torch.full((batch, n, k), float("nan"), dtype=torch.bfloat16, device=device()),
                              workspace=dirty_workspace(batch, n, k))
    assert bool(torch.isfinite(out).all())
    for i in {0, batch // 2, batch - 1}:
        ref.check_update(out[i], *ref.orthogonalize(g[i].double(), steps=steps), (n, k, i))
    assert torch.equal(fg.fg_orthogonalize(g, steps=steps), out)


@pytest.mark.parametrize("shape", [(96, 200), (3, 200, 64), (1500, 1300)])
def test_update_in_place(shape):
    """A bf16 gradient that its own update replaces."""
    g = torch.stack([gradient(i, *shape[-2:], torch.bfloat16) for i in range(shape[0])]) if len(shape) == 3 else gradient(1, *shape, torch.bfloat16)
    want = fg.fg_orthogonalize(g)
    assert fg.fg_orthogonalize(g, out=g) is g and torch.equal(g, want)


@pytest.mark.parametrize("batch,n,k", [(1, 64, 8192), (2, 76, 16200), (3, 5000, 130), (1, 33, 3003), (4, 60, 4200), (1, 309, 4853), (1, 700, 8192),
                                       (2, 3973, 496), (1, 856, 11323), (1, 1024, 16384), (1, 8200, 1500), (2, 1024, 8192),
                                       (1, 2048, 16384), (1, 2000, 18000), (2, 2048, 8192)])
def test_update_of_few_rows(batch, n, k):
    """Long contractions that several workgroups share, as far as the workspace has room for their sums."""
    g = torch.stack([gradient(i, n, k) for i in range(batch)])
    out = fg.fg_orthogonalize(g, out=torch.full((batch, n, k), float("nan"), dtype=torch.bfloat16, device=device()),
                              workspace=dirty_workspace(batch, n, k))
    for i in range(batch):
        ref.check_update(out[i], *ref.orthogonalize(g[i].double()), (n, k, i))
    for _ in range(3):
        assert torch.equal(fg.fg_orthogonalize(g), out)
    assert torch.equal(fg.fg_orthogonalize(g.flip(0)).flip(0), out)


def test_update_special_matrices():
    """Zeros give zeros, whatever stands beside; a NaN or an infinity stays in its own matrix; scales far from one do not matter."""
    g = torch.stack([gradient(i, 100, 150) for i in range(5)])
    want = fg.fg_orthogonalize(g)
    bad = g.clone()
    bad[0] = 0
    bad[1, 7, 9] = float("nan")
    bad[2, 0, 0] = float("inf")
    bad[3] *= 2.0 ** 60
    got = fg.fg_orthogonalize(bad)
    assert not got[0].any() and bool(torch.isnan(got[1:3]).all())
    assert torch.equal(got[3], fg.fg_orthogonalize(g[3:4] * 2.0 ** 40)[0])     # both far above eps
    assert torch.equal(got[4], want[4])
    tiny = fg.fg_orthogonalize(g[4] * 2.0 ** -100, eps=1e-38)
    ref.check_update(tiny, *ref.orthogonalize(g[4].double()))


def test_update_of_one_direction():
    """A rank-one gradient: p^5(1) u v^T along its direction; its empty directions carry the raised roundings."""
    u, v = rand(1, 300, 1), rand(2, 1, 500)
    g = u @ v
    want, err = ref.orthogonalize(g.double())
    ref.check_update(fg.fg_orthogonalize(g), want, err)


# ---- together -----------------------------------------------------------------------------------------

def test_training_step_of_a_linear():
    """norm -> Fprop; Dgrad -> norm's backward, Wgrad -> orthogonalised update -> the next step's weight codes. The FP8 GEMMs
    are the library's own; the operators are held to their definitions on what they are given."""
    rows, h, f = 256, 512, 384
    x, gamma = rows_like(1, rows, h, torch.bfloat16), 1 + rand(2, h, std=0.2)
    w = rand(3, f, h, std=h ** -0.5)
    n = fg.fg_norm_quantize(x, gamma, kind=fg.FG_NORM_RMS, eps=1e-6, token_tiles=True)
    check_norm(n, x, gamma, None, False, 1e-6, False, "step")
    wq, sw = fg.fg_quantize_w_128x128(w.bfloat16())
    y = fg.fg_fp8_gemm_fprop(n.q_cols, n.s_cols, wq, sw)
    values = ffn_ref.rows_values(n.q_cols, n.s_cols) @ ffn_ref.block_values(wq, sw).t()
    assert float((y.double() - values).abs().max()) <= 1e-2 * float(values.abs().max())
    dy = rand(4, rows, f, std=1e-3, dtype=torch.bfloat16)
    dyq, sdy, dytq, sdyt = fg.fg_quantize_act_1x128_both(dy)
    dn = fg.fg_fp8_gemm_dgrad(dyq, sdy, wq, sw)
    r = fg.fg_norm_bwd(x, None, n.rstd, gamma, dn, residual_grad=dn.bfloat16(), kind=fg.FG_NORM_RMS)
    check_grad(r, x, None, n.rstd, gamma, dn, dn.bfloat16(), False, "step")
    dw = fg.fg_fp8_gemm_wgrad(dytq, sdyt, n.q_rows, n.s_rows)
    u = fg.fg_orthogonalize(dw, scale=0.2 * max(f, h) ** 0.5)
    ref.check_update(u, *ref.orthogonalize(dw.double(), scale=0.2 * max(f, h) ** 0.5))
    w = w - 0.02 * u.float()
    wq2, _ = fg.fg_quantize_w_128x128(w.bfloat16())
    assert not torch.equal(wq, wq2)
