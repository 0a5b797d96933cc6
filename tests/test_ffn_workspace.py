"""Workspace sizes of the mixture of experts for any width: asked of the library itself, and their arithmetic under
sanitizers."""
import os
import shutil
import subprocess
import sys

import pytest

import fp8_fine_grained_amax_amd as fg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process of its own: an integer division by zero in the library would end the one it runs in.
ANY_WIDTH = """
import fp8_fine_grained_amax_amd as fg
query = fg.lib().fg_moe_few_tokens_workspace
for T in (0, 1, 4, 16, 17, 64):
    for topk in (1, 2, 32):
        for H in (*range(0, 130), 192, 255, 256, 1000, 4096, 4100, (1 << 20) - 1):
            for I in (0, 1, 31, 127, 128, 200, 256, 2048):
                size = query(T, topk, H, I)
                served = H % 128 == 0 and I % 128 == 0
                assert size >= T * topk * I * 4 if served else size == 0, (T, topk, H, I, size)
                assert size % 16 == 0 or not served, (T, topk, H, I, size)
print("every width asked")
"""


def test_moe_workspace_of_any_width():
    if not os.path.exists(fg.LIB_PATH):
        from fp8_fine_grained_amax_amd import build
        build.build()
    r = subprocess.run([sys.executable, "-c", ANY_WIDTH], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "every width asked" in r.stdout, (r.returncode, r.stdout, r.stderr)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_moe_workspace_under_sanitizers(tmp_path):
    exe = tmp_path / "moe_workspace_driver"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                        "-I", os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc"),
                        os.path.join(ROOT, "tests", "moe_workspace_driver.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout + r.stderr
    assert "moe workspace driver done" in r.stdout
