"""Host side of the training-step operators without a GPU: exports, argument checks with the documented status codes before any
HIP call, workspace sizes, the binding's refusals, and the checks' own arithmetic under sanitizers."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from fp8_fine_grained_amax_amd import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
A, B = 1 << 20, 2 << 20          # fake, aligned "device" addresses: never dereferenced on these paths
ODD = (1 << 20) + 4
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fg.LIB_PATH):
        from fp8_fine_grained_amax_amd import build
        build.build()
    return fg.lib()


def test_exports_every_declared_symbol(L):
    text = open(os.path.join(ROOT, "include", "fp8fg_train.h")).read()
    names = sorted(set(re.findall(r"^\s*(?:fg_status|int64_t)\s+(fg_\w+)\s*\(", text, re.M)))
    assert names == ["fg_norm_bwd", "fg_norm_bwd_workspace", "fg_norm_quantize", "fg_orthogonalize", "fg_orthogonalize_workspace"]
    for n in names:
        assert hasattr(L, n), n


def test_norm_rejections(L):
    def f(x=A, xt=1, ld=256, rows=128, cols=256, kind=0, gamma=A, beta=A, wt=0, eps=1e-5, mode=0, qc=B, sc=B, qr=B, sr=B, y=B,
          mean=B, rstd=B):
        return L.fg_norm_quantize(x, xt, ld, rows, cols, kind, gamma, beta, wt, eps, mode, qc, sc, qr, sr, y, mean, rstd, None)
    assert f(rows=-1) == INVALID and f(cols=-128) == INVALID and f(ld=255) == INVALID and f(xt=2) == INVALID
    assert f(wt=-1) == INVALID and f(kind=2) == INVALID and f(mode=2) == INVALID
    assert f(eps=0.0) == INVALID and f(eps=-1e-5) == INVALID and f(eps=INF) == INVALID and f(eps=NAN) == INVALID
    assert f(x=None) == INVALID and f(gamma=None) == INVALID and f(qc=None) == INVALID and f(sc=None) == INVALID
    assert f(qr=None) == INVALID and f(sr=None) == INVALID                        # halves of a pair
    assert f(rstd=None) == INVALID and f(mean=None) == INVALID                    # the tiles along the rows take them
    assert f(cols=200) == SHAPE and f(cols=18560, ld=18560) == SHAPE and f(rows=200) == SHAPE and f(rows=(1 << 25) + 128) == SHAPE
    assert f(rows=1 << 25, cols=2048, ld=2048) == SHAPE and f(ld=1 << 41) == SHAPE
    assert f(x=ODD) == MISALIGNED and f(ld=260) == MISALIGNED and f(xt=0, ld=258) == MISALIGNED and f(gamma=ODD) == MISALIGNED
    assert f(beta=ODD) == MISALIGNED and f(qc=ODD) == MISALIGNED and f(qr=ODD) == MISALIGNED and f(y=ODD) == MISALIGNED
    assert f(sc=B + 2) == MISALIGNED and f(sr=B + 2) == MISALIGNED and f(mean=B + 2) == MISALIGNED and f(rstd=B + 2) == MISALIGNED
    assert f(rows=0, x=None, qc=None) == OK and f(cols=0, ld=0, x=None) == OK


def test_norm_backward_rejections(L):
    need = L.fg_norm_bwd_workspace(600, 256)

    def f(x=A, xt=1, ldx=256, mean=A, rstd=A, gamma=A, wt=0, dy=A, dyt=0, lddy=256, dres=None, rt=0, ldr=256, rows=600, cols=256, kind=0,
          dx=B, dxt=0, dg=B, db=B, acc=0, ws=B, nws=need):
        return L.fg_norm_bwd(x, xt, ldx, mean, rstd, gamma, wt, dy, dyt, lddy, dres, rt, ldr, rows, cols, kind, dx, dxt, dg, db, acc, ws,
                             nws, None)
    assert f(rows=-1) == INVALID and f(cols=-128) == INVALID and f(ldx=255) == INVALID and f(lddy=100) == INVALID
    assert f(xt=2) == INVALID and f(wt=2) == INVALID and f(dyt=3) == INVALID and f(dxt=-1) == INVALID and f(kind=-1) == INVALID
    assert f(acc=2) == INVALID and f(nws=-1) == INVALID and f(dres=A, rt=2) == INVALID and f(dres=A, ldr=255) == INVALID
    assert f(x=None) == INVALID and f(mean=None) == INVALID and f(rstd=None) == INVALID and f(gamma=None) == INVALID
    assert f(dy=None) == INVALID and f(dx=None) == INVALID and f(ws=None) == INVALID and f(nws=need - 1) == INVALID
    assert f(dx=A, dy=B) == INVALID and f(dx=A, x=B) == INVALID                   # dx in place of x or dy
    assert f(dres=B, rt=1, dxt=0) == INVALID and f(dres=B, ldr=264) == INVALID     # dx as its own addend, laid out otherwise
    assert f(cols=200) == SHAPE and f(cols=18560, ldx=18560, lddy=18560) == SHAPE and f(rows=(1 << 25) + 1) == SHAPE
    assert f(ldx=1 << 41) == SHAPE and f(lddy=1 << 41) == SHAPE and f(dres=A, ldr=1 << 41) == SHAPE
    assert f(x=ODD) == MISALIGNED and f(ldx=260) == MISALIGNED and f(dy=ODD) == MISALIGNED and f(lddy=258) == MISALIGNED
    assert f(dres=ODD) == MISALIGNED and f(dres=A, rt=1, ldr=260) == MISALIGNED and f(dx=ODD) == MISALIGNED
    assert f(gamma=ODD) == MISALIGNED and f(dg=B + 2) == MISALIGNED and f(db=B + 1) == MISALIGNED and f(ws=B + 4) == MISALIGNED
    assert f(cols=0, ldx=0, lddy=0, x=None) == OK
    assert f(rows=0, x=None, dy=None, dx=None, dg=None, db=None) == OK and f(rows=0, x=None, acc=1) == OK


def test_update_rejections(L):
    need = L.fg_orthogonalize_workspace(2, 64, 100)

    def f(g=A, gt=0, ld=100, batch=2, n=64, k=100, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, scale=1.0, out=B, ws=B, nws=need):
        return L.fg_orthogonalize(g, gt, ld, batch, n, k, steps, a, b, c, eps, scale, out, ws, nws, None)
    assert f(batch=-1) == INVALID and f(n=-1) == INVALID and f(k=-1) == INVALID and f(ld=99) == INVALID and f(gt=2) == INVALID
    assert f(steps=0) == INVALID and f(steps=33) == INVALID and f(eps=0.0) == INVALID and f(eps=NAN) == INVALID
    assert f(scale=INF) == INVALID and f(a=NAN) == INVALID and f(b=INF) == INVALID and f(nws=need - 1) == INVALID
    assert f(g=None) == INVALID and f(out=None) == INVALID and f(ws=None) == INVALID
    # iterations that leave fp16's range
    assert f(a=6.0) == INVALID and f(b=-31.0) == INVALID and f(a=3.0, b=0.0, c=0.0, steps=2) == INVALID and f(c=1e30) == INVALID
    assert f(n=65537) == SHAPE and f(k=1 << 20, ld=1 << 20) == SHAPE and f(batch=1 << 30) == SHAPE and f(ld=1 << 41) == SHAPE
    assert f(g=A + 2) == MISALIGNED and f(gt=1, g=A + 1) == MISALIGNED and f(out=B + 1) == MISALIGNED and f(ws=B + 128) == MISALIGNED
    assert f(batch=0, g=None) == OK and f(n=0, g=None, out=None) == OK and f(k=0, ld=0, ws=None, nws=0) == OK


def test_workspace_sizes(L):
    w = L.fg_norm_bwd_workspace
    assert w(0, 256) == 0 and w(-1, 256) == 0 and w(4, 200) == 0 and w(4, 18560) == 0 and w(1 << 40, 256) == 0
    assert w(1, 128) == w(512, 18432) == 0 < w(513, 128) <= w(4096, 128) and w(1 << 25, 18432) <= 2 * 256 * 18432 * 4
    o = L.fg_orthogonalize_workspace
    assert o(0, 8, 8) == 0 and o(1, 0, 8) == 0 and o(1, 65537, 8) == 0 and o(1 << 40, 8, 8) == 0 and o(1, -5, 8) == 0
    assert o(1, 100, 200) == o(1, 200, 100) and o(1, 64, 64) < o(2, 64, 64) < o(2, 64, 128)
    assert o(1, 65536, 65536) >= 4 * 2 * 65536 ** 2


@pytest.fixture(scope="module")
def module():
    if not os.path.exists(os.path.join(os.path.dirname(ffn.__file__), "_ffn.so")):
        from fp8_fine_grained_amax_amd import build
        build.build()
    return ffn._ffn()


def test_arguments_are_counted(module):
    for f in (module.norm_quantize, module.norm_bwd, module.orthogonalize):
        with pytest.raises(TypeError, match="expected"):
            f(1)


@pytest.mark.parametrize("what", [None, 3, "x", torch.zeros(4, 128)])
def test_anything_but_a_gpu_tensor_is_refused(module, what):
    for call in (lambda: fg.fg_norm_quantize(what, what), lambda: fg.fg_norm_bwd(what, what, what, what, what),
                 lambda: fg.fg_orthogonalize(what)):
        with pytest.raises(fg.Fp8fgError):
            call()


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the HIP headers")
def test_host_layer_under_sanitizers(tmp_path):
    exe = tmp_path / "train_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc"),
           os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc", "train_api.cpp"),
           os.path.join(ROOT, "tests", "train_host_driver.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout + r.stderr
    assert "train host driver done" in r.stdout
