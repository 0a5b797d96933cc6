"""Host side of the feed-forward operators without a GPU: exports, argument checks with the documented status codes
before any HIP call, workspace sizes, and the checks' own arithmetic under sanitizers."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import fp8_fine_grained_amax_amd as fg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
A, B = 1 << 20, 2 << 20          # fake, aligned "device" addresses: never dereferenced on these paths
ODD = (1 << 20) + 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fg.LIB_PATH):
        from fp8_fine_grained_amax_amd import build
        build.build()
    return fg.lib()


def test_exports_every_declared_symbol(L):
    text = open(os.path.join(ROOT, "include", "fp8fg_ffn.h")).read()
    names = sorted(set(re.findall(r"^\s*(?:fg_status|int64_t)\s+(fg_\w+)\s*\(", text, re.M)))
    assert len(names) == 6, names
    for n in names:
        assert hasattr(L, n), n


def test_linear_rejections(L):
    def f(xq=A, sx=A, wq=A, sw=A, M=8, N=128, K=128, bias=None, bt=0, act=0, res=None, rt=0, ld=128, y=B, out=0, mode=0):
        return L.fg_fp8_gemm_fprop_epilogue(xq, sx, wq, sw, M, N, K, bias, bt, act, res, rt, ld, y, out, mode, None)
    assert f(M=-1) == INVALID and f(N=-1) == INVALID and f(K=-128) == INVALID
    assert f(mode=2) == INVALID and f(out=2) == INVALID and f(act=4) == INVALID and f(act=-1) == INVALID
    assert f(bias=A, bt=2) == INVALID and f(res=A, rt=-1) == INVALID and f(res=A, ld=127) == INVALID
    assert f(y=None) == INVALID and f(wq=None) == INVALID
    assert f(res=B, rt=1, out=0) == INVALID and f(res=B, ld=256) == INVALID         # y as its own residual, laid out otherwise
    assert f(K=100) == SHAPE and f(K=(1 << 24) + 128) == SHAPE and f(M=1 << 40, N=1 << 30, ld=1 << 30) == SHAPE
    assert f(res=A, ld=1 << 41) == SHAPE
    assert f(xq=ODD) == MISALIGNED and f(y=ODD) == MISALIGNED and f(bias=A + 2) == MISALIGNED
    assert f(bias=A + 1, bt=1) == MISALIGNED and f(res=A + 2) == MISALIGNED and f(sw=A + 2) == MISALIGNED
    assert f(M=0, xq=None, y=None) == OK and f(N=0, ld=0, y=None) == OK


def test_act_forward_rejections(L):
    def f(z=A, rows=4, F=128, ld=256, act=3, gated=1, mode=0, zq=B, sz=B, aq=B, sa=B):
        return L.fg_act_checkpoint_fwd(z, rows, F, ld, act, gated, mode, zq, sz, aq, sa, None)
    assert f(rows=-1) == INVALID and f(F=-128) == INVALID and f(act=7) == INVALID and f(gated=2) == INVALID
    assert f(mode=3) == INVALID and f(ld=128) == INVALID and f(z=None) == INVALID and f(sa=None) == INVALID
    assert f(F=192, ld=384) == SHAPE and f(F=1 << 31, ld=1 << 33) == SHAPE and f(rows=1 << 31) == SHAPE
    assert f(F=(1 << 23) + 128, ld=1 << 25) == SHAPE and f(rows=(1 << 25) + 1) == SHAPE
    assert f(rows=1 << 25, F=1 << 23, ld=1 << 25) == SHAPE                          # more workgroups than a launch has
    assert f(z=ODD) == MISALIGNED and f(ld=260) == MISALIGNED and f(zq=ODD) == MISALIGNED and f(sz=B + 2) == MISALIGNED
    assert f(rows=0, z=None, zq=None) == OK and f(F=0, ld=0, z=None) == OK


def test_act_backward_rejections(L):
    def f(zq=A, sz=A, da=A, dt=0, ld=128, rows=256, F=128, act=3, gated=1, mode=0, qc=B, sc=B, qr=B, sr=B, ar=B, sa=B,
          db=B, ws=B, nws=2 * 256 * 4):
        return L.fg_act_checkpoint_bwd(zq, sz, da, dt, ld, rows, F, act, gated, mode, qc, sc, qr, sr, ar, sa, db, ws, nws, None)
    assert f(rows=-1) == INVALID and f(F=-1) == INVALID and f(ld=127) == INVALID and f(act=4) == INVALID
    assert f(dt=2) == INVALID and f(gated=-1) == INVALID and f(mode=2) == INVALID and f(nws=-1) == INVALID
    assert f(zq=None) == INVALID and f(da=None) == INVALID and f(qc=None) == INVALID
    assert f(qr=None) == INVALID and f(sr=None) == INVALID and f(ar=None) == INVALID and f(sa=None) == INVALID   # halves of a pair
    assert f(ws=None) == INVALID and f(nws=2 * 256 * 4 - 1) == INVALID
    assert f(rows=200) == SHAPE and f(F=100) == SHAPE and f(F=1 << 31, ld=1 << 31) == SHAPE and f(rows=1 << 31) == SHAPE
    assert f(F=(1 << 23) + 128, ld=1 << 23) == INVALID and f(ld=(1 << 23) + 4) == SHAPE and f(rows=(1 << 25) + 128) == SHAPE
    assert f(rows=200, qr=None, sr=None) == SHAPE                                   # a along the rows alone
    assert f(zq=ODD) == MISALIGNED and f(ld=130) == MISALIGNED and f(dt=1, ld=132) == MISALIGNED and f(db=B + 2) == MISALIGNED
    assert f(rows=0, zq=None, sz=None, da=None, qc=None, sc=None, db=None) == OK and f(F=0, ld=0, zq=None) == OK


def test_moe_rejections(L):
    def f(x=A, ldx=256, ids=A, w=A, T=4, topk=2, w1=A, s1=A, w2=A, s2=A, E=8, H=256, I=128, act=3, mode=0, ws=A,
          nws=1 << 20, y=B, ldy=256, out=1):
        return L.fg_moe_few_tokens(x, ldx, ids, w, T, topk, w1, s1, w2, s2, E, H, I, act, mode, ws, nws, y, ldy, out, None)
    assert f(T=-1) == INVALID and f(topk=0) == INVALID and f(E=0) == INVALID and f(ldx=255) == INVALID and f(ldy=128) == INVALID
    assert f(act=4) == INVALID and f(mode=2) == INVALID and f(out=2) == INVALID and f(nws=-1) == INVALID
    assert f(ids=None) == INVALID and f(w1=None) == INVALID and f(y=None) == INVALID and f(ws=None) == INVALID
    assert f(nws=4 * 2 * 128 * 4 - 1) == INVALID
    assert f(T=65) == SHAPE and f(topk=33) == SHAPE and f(E=2049) == SHAPE and f(H=192) == SHAPE and f(I=100) == SHAPE
    assert f(H=(1 << 20) + 128, ldx=1 << 21, ldy=1 << 21) == SHAPE and f(I=(1 << 20) + 128) == SHAPE
    assert f(x=ODD) == MISALIGNED and f(ldx=260) == MISALIGNED and f(y=ODD) == MISALIGNED and f(ws=ODD) == MISALIGNED
    assert f(ids=A + 2) == MISALIGNED
    assert f(T=0, x=None, ids=None) == OK and f(H=0, x=None) == OK


def test_workspace_sizes(L):
    w = L.fg_act_checkpoint_bwd_workspace
    assert w(128, 256, 0) == 0 and w(0, 256, 1) == 0 and w(129, 256, 0) == 2 * 256 * 4 and w(256, 256, 1) == 2 * 512 * 4
    assert w(-1, 256, 0) == 0 and w(1 << 40, 256, 0) == 0
    m = L.fg_moe_few_tokens_workspace
    assert m(4, 2, 256, 128) == 4 * 2 * 128 * 4 and m(0, 2, 256, 128) == 0 and m(65, 2, 256, 128) == 0
    # more tokens: the plan and the activations' codes besides the hidden values; never less for more of anything
    rows = 64 * 8
    assert m(64, 8, 7168, 2048) > rows * 2048 * 5 + 64 * 7168
    for a, b in (((16, 8, 1024, 512), (17, 8, 1024, 512)), ((17, 2, 256, 128), (64, 2, 256, 128)), ((64, 2, 256, 128), (64, 32, 256, 128)),
                 ((64, 8, 2048, 1024), (64, 8, 2048, 2048))):
        assert m(*a) < m(*b), (a, b)


def test_launches_past_32_bits_of_threads_are_refused(L):
    def fwd(rows, F):
        return L.fg_act_checkpoint_fwd(A, rows, F, 2 * F, 3, 1, 0, B, B, B, B, None)
    def bwd(rows, F):
        return L.fg_act_checkpoint_bwd(A, A, A, 0, F, rows, F, 3, 1, 0, B, B, None, None, None, None, None, None, 0, None)
    def moe(T, topk, E, I):
        return L.fg_moe_few_tokens(A, 256, A, A, T, topk, A, A, A, A, E, 256, I, 3, 0, None, 0, B, 256, 1, None)
    assert fwd(1 << 25, 2048) == SHAPE and fwd(1 << 25, 1 << 23) == SHAPE
    assert bwd(1 << 25, 4096) == SHAPE and bwd((1 << 25) - 5, 4096) == SHAPE
    assert moe(64, 32, 2048, 1 << 18) == SHAPE and moe(16, 32, 512, 1 << 20) == SHAPE
    assert moe(64, 32, 2048, (1 << 18) - 128) == INVALID and moe(64, 32, 256, 1 << 20) == INVALID    # no workspace: within limits


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(4, 256, dtype=torch.bfloat16)
    u = torch.zeros(4, 256, dtype=torch.uint8)
    s = torch.zeros(2, 4)
    with pytest.raises(fg.Fp8fgError):
        fg.fg_act_checkpoint_fwd(z, fg.FG_ACT_SILU)
    with pytest.raises(fg.Fp8fgError):
        fg.fg_act_checkpoint_bwd(u, s, z, fg.FG_ACT_SILU)
    with pytest.raises(fg.Fp8fgError):
        fg.fg_fp8_gemm_fprop_epilogue(u, s, u, s)
    with pytest.raises(fg.Fp8fgError):
        fg.fg_moe_few_tokens(z, u, s, u, s, u, s)


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the HIP headers")
def test_host_layer_under_sanitizers(tmp_path):
    exe = tmp_path / "ffn_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc"),
           os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc", "ffn_api.cpp"),
           os.path.join(ROOT, "tests", "ffn_host_driver.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout + r.stderr
    assert "ffn host driver done" in r.stdout
