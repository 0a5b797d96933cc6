"""Calls of the training-step operators that their documentation allows or refuses, beside the sizes of test_gpu_train.py: captured
graphs, several streams and threads, tensors past 2^32 bytes, malformed arguments."""
import threading

import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from tests import train_ref as ref
from tests.gpu_util import device
from tests.test_gpu_ffn_large import repeated, same_blocks
from tests.test_gpu_train import check_grad, check_norm, grad_case, gradient, rand, rows_like

pytestmark = pytest.mark.gpu


def outputs(x, gamma, beta, mean, rstd, dy, g):
    """Every operator once: a flat list of tensors."""
    n = fg.fg_norm_quantize(x, gamma, beta, token_tiles=True, with_y=True)
    r = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=dy, bias_grad=True)
    return [*n, *r, fg.fg_orthogonalize(g), fg.fg_orthogonalize(g[:70, :90], steps=2)]


def case(seed, rows=256, cols=896, n=300, k=200):
    x, mean, rstd, gamma, dy = grad_case(rows, cols, True)
    return [x + rand(seed, rows, cols, std=0.01).to(x.dtype), gamma, rand(seed + 1, cols), mean, rstd, dy * (1 + seed), gradient(seed, n, k)]


def test_two_graphs_of_one_pool():
    """Two captures whose workspaces lie in the same memory, replayed in turn with eager work and new inputs between."""
    ins = [case(1), case(2, 384, 2048, 140, 600)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a in ins:
            outputs(*a)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        outs = [outputs(*ins[0])]
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        outs.append(outputs(*ins[1]))
    for k in range(4):
        for i, a in enumerate(ins):
            for t, new in zip(a, case(10 * k + i, *a[0].shape, *a[6].shape)):
                t.copy_(new)
        for graph, out, a in zip(graphs, outs, ins):
            graph.replay()
            want = outputs(*a)
            torch.cuda.synchronize()
            for i, (got, w) in enumerate(zip(out, want)):
                assert torch.equal(got.view(torch.uint8), w.view(torch.uint8)), (k, i)


def test_streams_and_threads():
    """Four threads, each on a stream of its own, several calls each: the same as one after the other, bit for bit."""
    ins = [case(i, 128 + 128 * i, 512, 200 + 50 * i, 260) for i in range(4)]
    want = [outputs(*a) for a in ins]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    out = outputs(*ins[i])
            stream.synchronize()
            got[i] = out
        except Exception as e:          # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(want, got):
        for i, (p, q) in enumerate(zip(a, b)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), i


def test_runs_are_equal():
    a = case(5, 1000 // 128 * 128, 1024, 900, 520)
    first = outputs(*a)
    for _ in range(3):
        for p, q in zip(first, outputs(*a)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


# ---- past 2^32 bytes ----------------------------------------------------------------------------------

@pytest.mark.parametrize("cols,times,tokens", [(16384, 1094, True), (18432, 1000, False), (1024, 17000, True)])
def test_norm_past_32_bits(cols, times, tokens):
    x = rows_like(1, 128, cols, torch.bfloat16)
    gamma, beta = 1 + rand(2, cols, std=0.2), rand(3, cols, std=0.1)
    # enough rows for the same kernel as the large run's
    small = fg.fg_norm_quantize(repeated(x, 3), gamma, beta, token_tiles=tokens)
    check_norm(small, repeated(x, 3), gamma, beta, True, 1e-5, False, cols)
    big = fg.fg_norm_quantize(repeated(x, times), gamma, beta, token_tiles=tokens)
    names = [("q_cols", 0), ("s_cols", 1), ("mean", 0), ("rstd", 0)] + ([("q_rows", 1), ("s_rows", 0)] if tokens else [])
    for name, dim in names:
        part = getattr(small, name).narrow(dim, 0, 1 if name == "s_rows" else 128).contiguous()
        assert same_blocks(getattr(big, name), part, dim), name


def test_norm_backward_past_32_bits():
    cols, times = 16384, 1094
    x, mean, rstd, gamma, dy = grad_case(128, cols, True)
    small = fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=dy, bias_grad=True)
    check_grad(small, x, mean, rstd, gamma, dy, dy, True, "small")
    big = fg.fg_norm_bwd(repeated(x, times), mean.repeat(times), rstd.repeat(times), gamma, repeated(dy, times),
                         residual_grad=repeated(dy, times), bias_grad=True)
    assert same_blocks(big.dx, small.dx)
    rows = 128 * times
    # additions of a column as in check_grad: their number times half a step, of the sum of magnitudes
    _, _, dg, db, dg_abs, db_abs = ref.norm_grad(x.double(), mean.double(), rstd.double(), gamma.double(), dy.double(), None, True)
    for got, want, mag in ((big.dgamma, dg, dg_abs), (big.dbeta, db, db_abs)):
        assert bool(((got.double() - times * want).abs() <= (rows / 256 + 53) * 2.0 ** -24 * times * mag).all())


def test_update_of_a_matrix_past_32_bits():
    """A block-diagonal gradient of 46080 x 46080 (8.5 GB): every block's update is its own, by the whole matrix's norm."""
    side, block = 46080, 512
    g = torch.zeros(side, side, device=device())
    blocks = {}
    for i in (0, 1, 7, 44, 60, 89):
        blocks[i] = gradient(i, block, block)
        g[i * block:(i + 1) * block, i * block:(i + 1) * block] = blocks[i]
    norm = sum(float(b.double().square().sum()) for b in blocks.values()) ** 0.5
    out = fg.fg_orthogonalize(g, steps=2)
    del g
    for i, b in blocks.items():
        at = slice(i * block, (i + 1) * block)
        own = float(torch.linalg.matrix_norm(b.double()))
        # the block's norm stands for the whole one's through eps
        ref.check_update(out[at, at], *ref.orthogonalize(b.double(), steps=2, eps=norm - own), i)
        out[at, at] = 0
    assert not any(bool(part.any()) for part in out.split(4096))


def test_update_of_a_batch_past_32_bits():
    b, n, k = 40, 2100, 13000
    g = torch.empty(b, n, k, device=device())
    for i in range(b):
        g[i] = gradient(i % 3, n, k, tokens=2200)
    out = fg.fg_orthogonalize(g, steps=1)
    for i in range(3):
        ref.check_update(out[i], *ref.orthogonalize(g[i].double(), steps=1), i)
    for i in range(3, b):                    # the same matrix, whatever tiles it falls on
        assert torch.equal(out[i], out[i % 3]), i


# ---- refusals -----------------------------------------------------------------------------------------

def refused(call, match=None):
    with pytest.raises(fg.Fp8fgError, match=match):
        call()
    assert fg.lib().fg_last_hip_error() == 0


def test_norm_refusals():
    x, gamma = rows_like(1, 130, 256, torch.bfloat16), torch.ones(256, device=device())
    half = torch.ones(256, device=device(), dtype=torch.float16)
    refused(lambda: fg.fg_norm_quantize(x[0], gamma), "dimensions")
    refused(lambda: fg.fg_norm_quantize(x.half(), gamma), "float32 or bfloat16")
    refused(lambda: fg.fg_norm_quantize(x, half), "gamma")
    refused(lambda: fg.fg_norm_quantize(x, gamma[:128]), "gamma")
    refused(lambda: fg.fg_norm_quantize(x, gamma, gamma.bfloat16()), "beta")
    refused(lambda: fg.fg_norm_quantize(x, gamma.cpu()), "GPU")
    refused(lambda: fg.fg_norm_quantize(x.t(), gamma), "gamma|stride")
    refused(lambda: fg.fg_norm_quantize(x[:1].expand(130, 256), gamma), "overlap")
    refused(lambda: fg.fg_norm_quantize(x, gamma, kind=2), "norm")
    refused(lambda: fg.fg_norm_quantize(x, gamma, eps=0.0), "invalid")
    refused(lambda: fg.fg_norm_quantize(x, gamma, token_tiles=True), "shape")
    refused(lambda: fg.fg_norm_quantize(x[:, :200], gamma[:200]), "shape")
    refused(lambda: fg.fg_norm_quantize(torch.ones(2, 18560, device=device()), torch.ones(18560, device=device())), "shape")
    refused(lambda: fg.fg_norm_quantize(x[:, 1:129], gamma[:128].clone()), "misaligned")
    good = fg.fg_norm_quantize(x, gamma, with_y=True)
    for name in ("q_cols", "s_cols", "y", "mean", "rstd"):
        bad = good._replace(**{name: getattr(good, name)[:-1]})
        refused(lambda: fg.fg_norm_quantize(x, gamma, with_y=True, out=bad), name)
    assert fg.fg_norm_quantize(x, gamma, out=good).y is None


def test_norm_backward_refusals():
    x, mean, rstd, gamma, dy = grad_case(130, 256, True)
    refused(lambda: fg.fg_norm_bwd(x, None, rstd, gamma, dy), "mean")
    refused(lambda: fg.fg_norm_bwd(x, mean[:-1], rstd, gamma, dy), "mean")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd.double(), gamma, dy), "rstd")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy[:-1]), "dy")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy.half()), "dy")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=dy[:, :128]), "residual_grad")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, out_dtype=torch.float16), "dtype")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, dx=dy[:-1]), "dx")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, accumulate=True), "accumulate")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, bias_grad=True, accumulate=True, dgamma=gamma.clone()), "accumulate")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, dx=dy), "invalid")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, dx=x), "invalid")
    more = grad_case(600, 256, True)
    refused(lambda: fg.fg_norm_bwd(*more, workspace=torch.empty(16, dtype=torch.uint8, device=device())), "invalid")
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, workspace=gamma), "uint8")
    wide = torch.zeros(130, 512, device=device())
    refused(lambda: fg.fg_norm_bwd(x, mean, rstd, gamma, dy, residual_grad=wide[:, :256], dx=wide[:, :256]), "dx")
    assert fg.fg_norm_bwd(x, mean, rstd, gamma, dy, weight_grad=False).dgamma is None


def test_update_refusals():
    g = gradient(1, 40, 60)
    refused(lambda: fg.fg_orthogonalize(g[0]), "dimensions")
    refused(lambda: fg.fg_orthogonalize(g[None, None]), "dimensions")
    refused(lambda: fg.fg_orthogonalize(g.half()), "float32 or bfloat16")
    refused(lambda: fg.fg_orthogonalize(g.t()), "stride")
    refused(lambda: fg.fg_orthogonalize(g[:1].expand(40, 60)), "overlap")
    refused(lambda: fg.fg_orthogonalize(torch.stack([g, g, g])[::2]), "one behind the other")
    refused(lambda: fg.fg_orthogonalize(g, steps=0), "steps")
    refused(lambda: fg.fg_orthogonalize(g, steps=33), "invalid")
    refused(lambda: fg.fg_orthogonalize(g, eps=0.0), "invalid")
    refused(lambda: fg.fg_orthogonalize(g, coefficients=(8.0, 0.0, 0.0)), "invalid")
    refused(lambda: fg.fg_orthogonalize(g, scale=float("inf")), "invalid")
    refused(lambda: fg.fg_orthogonalize(g, out=torch.empty(40, 60, device=device())), "out")
    refused(lambda: fg.fg_orthogonalize(g, workspace=torch.empty(1000, dtype=torch.uint8, device=device())), "invalid")
    refused(lambda: fg.fg_orthogonalize(torch.zeros(1, 65537, device=device())), "shape")
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 4)):
        out = fg.fg_orthogonalize(torch.empty(shape, device=device()))
        assert out.shape == shape and out.dtype == torch.bfloat16
    with pytest.raises(TypeError):
        fg.fg_orthogonalize(g, steps="five")
