"""What the build makes when the tools of the Python binding are missing or fail: the C
library, which needs none of them, all the same.  No compiler is run."""
import importlib.util
import os
import subprocess

import pytest

from exact_tiled_attention_40_b200 import build as b


class Run:
    """Stands for subprocess.run: writes the file behind -o, or fails for `broken`."""

    def __init__(self, broken=(), missing=()):
        self.broken, self.missing, self.outputs = broken, missing, []

    def __call__(self, cmd, **kw):
        tool = os.path.basename(cmd[0])
        if tool in self.missing:
            raise FileNotFoundError(cmd[0])
        if tool in self.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("built")
        self.outputs.append(os.path.basename(out))
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs under tmp_path."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "DEBUG_BUILD", str(tmp_path / "_build" / "debug"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "DEBUG_LIB", str(tmp_path / "_build" / "debug" / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_step.so"))
    return tmp_path


def use(monkeypatch, run, without=()):
    which = b.shutil.which
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b.shutil, "which", lambda n: None if n in without else which(n))


def test_both_are_built(tree, monkeypatch):
    run = Run()
    use(monkeypatch, run)
    assert b.build() == str(tree / "lib.so")
    assert (tree / "lib.so").exists() and (tree / "_step.so").exists()
    run.outputs.clear()
    b.build()                                    # nothing is stale
    assert run.outputs == []


def test_without_a_compiler_for_the_binding(tree, monkeypatch, capsys):
    use(monkeypatch, Run(missing=("g++",)), without=("g++",))
    assert b.build() == str(tree / "lib.so")
    assert (tree / "lib.so").exists() and not (tree / "_step.so").exists()
    assert "g++" in capsys.readouterr().err


def test_without_torch(tree, monkeypatch, capsys):
    use(monkeypatch, Run(broken=("g++",)))       # (no header to be found)
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda n, *a: None if n == "torch" else find(n, *a))
    assert b.build() == str(tree / "lib.so")
    assert (tree / "lib.so").exists() and not (tree / "_step.so").exists()
    assert "torch" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_fails_behind_the_library(tree, monkeypatch):
    use(monkeypatch, Run(broken=("g++",)))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert (tree / "lib.so").exists()


def test_a_library_that_does_not_compile_fails(tree, monkeypatch):
    use(monkeypatch, Run(broken=("nvcc",)))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        b.build()
    assert not (tree / "lib.so").exists()


def test_the_binding_is_rebuilt_for_another_torch(tree, monkeypatch):
    run = Run()
    use(monkeypatch, run)
    b.build()
    run.outputs.clear()
    monkeypatch.setattr(b, "binding_abi", lambda: "torch 0.0.1, another Python")
    b.build()
    assert run.outputs == ["_step.so"]
    run.outputs.clear()
    b.build()
    assert run.outputs == []


def test_the_build_is_for_the_running_torch_and_python():
    import sys
    import torch
    assert torch.__version__ in b.binding_abi() and sys.implementation.cache_tag in b.binding_abi()


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    from exact_tiled_attention_40_b200 import fa
    monkeypatch.setattr(fa, "_step", None)
    fa._native()                                 # (this tree's own loads)
    monkeypatch.setattr(fa, "_step", None)
    monkeypatch.setattr(fa, "binding_abi", lambda: "torch 0.0.1, another Python")
    with pytest.raises(fa.FAError, match="another Python"):
        fa._native()
    assert fa._step is None


def test_a_torch_that_does_not_say_its_version(tmp_path, monkeypatch):
    monkeypatch.setattr(b, "_torch_dir", lambda: str(tmp_path))
    assert "unknown" in b.binding_abi()
    (tmp_path / "version.py").write_text("git_version = 'x'\n")
    assert "unknown" in b.binding_abi()
    monkeypatch.setattr(b, "_torch_dir", lambda: None)
    assert "unknown" in b.binding_abi()
