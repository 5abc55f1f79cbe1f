"""The build's order (no compiler is run): the C library, which needs hipcc alone, is there whatever becomes of the
CPython module."""
import builtins
import os
import subprocess

import pytest

from bit_ternary_weight_bitlinear_amd import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Every command succeeds and leaves its output file, but g++ does what `compiler` says."""
    state = {"g++": 0}

    def run(cmd, **kw):
        status = state["g++"] if cmd[0] == "g++" else 0
        if status == 0:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, status, "", "no such header" if status else "")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name in ("LIB", "BENCH_LIB", "BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    state["dir"] = str(tmp_path)
    return state


def test_library_is_linked_when_the_binding_does_not_compile(fake):
    fake["g++"] = 1
    with pytest.raises(RuntimeError, match="no such header"):
        build.build(out_dir=fake["dir"])
    assert os.path.exists(build.LIB) and os.path.exists(build.BENCH_LIB) and not os.path.exists(build.BINDING)


def test_library_is_built_without_torch(fake, monkeypatch, capsys):
    real = builtins.__import__

    def no_torch(name, *args, **kw):
        if name == "torch":
            raise ImportError("No module named 'torch'")
        return real(name, *args, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert build.build(out_dir=fake["dir"]) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "_binding.so is not built" in capsys.readouterr().err


def test_everything_is_built(fake):
    assert build.build(out_dir=fake["dir"]) == build.LIB
    assert all(os.path.exists(p) for p in (build.LIB, build.BENCH_LIB, build.BINDING))
