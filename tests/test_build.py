"""What build.build() needs: the C library hipcc alone, the Python binding of the feed-forward operators torch and g++ too."""
import os
import subprocess
import sys

import pytest

from fp8_fine_grained_amax_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """build.build() with every command replaced by one that only leaves its output file; returns what was run."""
    ran = []

    def run(cmd, **kwargs):
        ran.append(cmd)
        if "-o" in cmd:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)
    for name in ("CSRC", "LIB", "FFN_MODULE", "C_CONSUMER"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    os.makedirs(build.CSRC)
    return ran


def compilers(ran):
    return {os.path.basename(c[0]) for c in ran} - {os.path.basename(sys.executable)}


def test_everything(commands):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.FFN_MODULE)
    assert compilers(commands) == {"hipcc", "g++"}


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_c_library_and_its_consumer_need_hipcc_only(commands, monkeypatch, capsys, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr("shutil.which", lambda name, *a, **k: None)
    open(build.FFN_MODULE, "w").close()                # an older build's, linked against another library
    assert build.build() == build.LIB
    assert build.build_c_consumer() == build.C_CONSUMER
    assert os.path.exists(build.LIB) and os.path.exists(build.C_CONSUMER) and not os.path.exists(build.FFN_MODULE)
    assert compilers(commands) == {"hipcc"}
    assert missing in capsys.readouterr().err          # said, not silent: the binding fails at its first use


def test_a_binding_that_does_not_compile_is_an_error(commands, monkeypatch):
    good = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **k: subprocess.CompletedProcess(cmd, 1, "", "no")
                        if cmd[0] == "g++" else good(cmd, **k))
    with pytest.raises(RuntimeError, match="ffn_binding"):
        build.build()
