"""The build's steps, without running a compiler: the library needs hipcc alone."""
import os
import sys

import pytest

from bit_quantized_gemv_amd import build


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """The output files of the build's commands, in their order."""
    done = []

    def run(cmd, what):
        if "-lqmv" in cmd:
            assert os.path.join(str(tmp_path), "libqmv.so") in done
        out = cmd[cmd.index("-o") + 1]
        done.append(out[:-4] if out.endswith(".tmp") else out)
        open(out, "w").close()

    for name in ("BUILD", "LIBDIR"):
        monkeypatch.setattr(build, name, str(tmp_path))
    for name, f in (("LIB", "libqmv.so"), ("PY", "qmv_ops_py.so")):
        monkeypatch.setattr(build, name, str(tmp_path / f))
    monkeypatch.setattr(build, "_run", run)
    return done


def names(done):
    return [os.path.basename(f) for f in done if f.endswith(".so")]


def test_library_then_binding(steps):
    assert build.build() == build.LIB
    assert names(steps) == ["libqmv.so", "qmv_ops_py.so"]


def test_without_torch(steps, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)          # what an import finds where there is none
    assert build.build() == build.LIB
    assert names(steps) == ["libqmv.so"]
    assert "torch" in capsys.readouterr().err


def test_without_a_host_compiler(steps, monkeypatch, capsys):
    monkeypatch.setenv("PATH", "")
    assert build.build() == build.LIB
    assert names(steps) == ["libqmv.so"]
    assert "g++" in capsys.readouterr().err


def test_a_binding_that_fails_leaves_the_library(steps, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed on ops_py.cpp")

    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="ops_py.cpp"):
        build.build()
    assert names(steps) == ["libqmv.so"] and os.path.exists(build.LIB)
