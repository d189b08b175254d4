"""The build's parts on the host, with compilers that only pretend: the library does not depend on the module for torch
tensors, whose failure is its own."""
import os
import subprocess
import warnings

import pytest

from zero_partitioned_mixed_flat_gb300 import _abi, build


class Compilers:
    """Commands in the place of nvcc and g++, which write an empty output; g++ may fail, or not be there."""

    def __init__(self):
        self.module, self.ran = "works", []

    def __call__(self, cmd, **_):
        self.ran.append(os.path.basename(cmd[0]))
        if cmd[0] == "g++":
            if self.module == "missing":
                raise FileNotFoundError(2, "No such file or directory", "g++")
            if self.module == "fails":
                return subprocess.CompletedProcess(cmd, 1, "", "fatal error: Python.h: No such file")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def take(self):
        ran, self.ran = self.ran, []
        return ran


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    tools = Compilers()
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("")
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libzero.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build, "TENSORS_ERROR", str(tmp_path / "_tensors.error"), raising=False)
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(torch_dir))
    monkeypatch.setattr(build.subprocess, "run", tools)
    return tools


@pytest.mark.parametrize("how", ["fails", "missing"])
def test_the_library_builds_without_the_module(compilers, how, monkeypatch):
    compilers.module = how
    with pytest.warns(RuntimeWarning, match="Python.h" if how == "fails" else "g\\+\\+"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)
    assert compilers.take().count("nvcc") == len(build._sources()) + 1
    # what needs the module says why there is none
    monkeypatch.setattr(_abi, "_TENSORS", None)
    monkeypatch.setattr(_abi, "load", lambda: None)
    monkeypatch.setattr(_abi, "LIB_PATH", build.LIB)
    with pytest.raises(ImportError, match="Python.h" if how == "fails" else "g\\+\\+"):
        _abi.tensors()
    # the next build tries the module alone
    compilers.module = "works"
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert build.build() == build.LIB
    assert compilers.take() == ["g++", "g++"]
    assert os.path.exists(build.TENSORS) and not os.path.exists(build.TENSORS_ERROR)
    build.build()
    assert compilers.take() == []


def test_a_stale_module_is_not_left_behind(compilers):
    build.build()
    assert os.path.exists(build.TENSORS)
    compilers.module = "fails"
    with pytest.warns(RuntimeWarning):
        build.build(force=True)
    assert os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)


def test_no_torch_no_module(compilers, monkeypatch):
    monkeypatch.setattr(build, "_torch_dir", lambda: None)
    build.build()
    assert "g++" not in compilers.take() and os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)
    build.build()
    assert compilers.take() == []


def test_a_library_that_fails_is_an_error(compilers, monkeypatch):
    def fail(cmd, **_):
        return subprocess.CompletedProcess(cmd, 1, "", "no")
    monkeypatch.setattr(build.subprocess, "run", fail)
    with pytest.raises(RuntimeError):
        build.build()
    assert not os.path.exists(build.LIB)
