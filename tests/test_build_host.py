"""What is built where torch is, and where it is not.  Compilers are stood in for: each "builds" an empty file."""
import importlib.util
import os
import subprocess

import pytest

from memory_bound_elementwise_gb300 import _build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """The products' folder and the commands that build() has run."""
    commands = []

    def run(cmd, **kwargs):
        out = cmd[cmd.index("-o") + 1]
        commands.append(cmd)
        if any(os.path.basename(c) in fails for c in cmd):
            return subprocess.CompletedProcess(cmd, 1, "error")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "")

    fails = set()
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libew.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_ew_torch.so"))
    monkeypatch.setattr(_build.subprocess, "run", run)
    return tmp_path, commands, fails


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_needs_no_torch(monkeypatch, built, capsys):
    folder, commands, _ = built
    without_torch(monkeypatch)
    assert _build.build() == str(folder / "libew.so")
    assert (folder / "libew.so").exists() and not (folder / "_ew_torch.so").exists()
    assert not any(_build.BINDING_SOURCE in c for c in commands)
    assert "torch" in capsys.readouterr().err
    n = len(commands)
    _build.build()
    assert len(commands) == n  # nothing is built twice


def test_torch_that_comes_later_adds_the_binding_alone(monkeypatch, built):
    folder, commands, _ = built
    with monkeypatch.context() as m:
        without_torch(m)
        _build.build()
    if _build._torch_dir() is None:
        pytest.skip("no torch here")
    commands.clear()
    _build.build()
    assert (folder / "_ew_torch.so").exists() and len(commands) == 2  # compiled, linked
    commands.clear()
    _build.build()
    assert not commands


def test_a_binding_that_does_not_compile_leaves_the_library(built):
    folder, _, fails = built
    if _build._torch_dir() is None:
        pytest.skip("no torch here")
    fails.add(os.path.basename(_build.BINDING_SOURCE))
    with pytest.raises(RuntimeError, match="ew_torch.cpp"):
        _build.build()
    assert (folder / "libew.so").exists()
