"""The library needs nvcc alone: the binding's extension is built after it, and whatever is missing for that costs
a warning."""
import os
import subprocess
import sys

import pytest

from attention_kl_divergence_02_b200 import build


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """Compilers that only write the file they are asked for; the list of what was asked for."""
    asked = []

    def check_call(cmd, *a, **kw):
        asked.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libstreamkl.so"))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    if hasattr(build, "FASTCALL"):
        monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    return asked


def kinds(asked):
    return ["extension" if any(x.endswith("fastcall.cpp") for x in cmd) else "library" for cmd in asked]


def test_the_library_comes_first(compiler):
    assert build.build(force=True) == build.LIB and os.path.exists(build.LIB)
    assert kinds(compiler)[0] == "library"


def test_without_torch(compiler, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="extension"):
        assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and kinds(compiler) == ["library"]


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, "g++"), FileNotFoundError("g++")])
def test_without_a_host_compiler_that_works(compiler, monkeypatch, error):
    pytest.importorskip("torch")
    works = build.subprocess.check_call

    def check_call(cmd, *a, **kw):
        if kinds([cmd]) == ["extension"]:
            raise error
        works(cmd)

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    with pytest.warns(UserWarning, match="extension"):
        assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB)


def test_a_library_that_does_not_build_is_an_error(compiler, monkeypatch):
    def check_call(cmd, *a, **kw):
        raise subprocess.CalledProcessError(1, cmd[0])
    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)


def test_an_extension_for_another_torch_is_not_taken(compiler, monkeypatch):
    """It belongs to the headers that it was compiled with: built again, and not loaded, for another version."""
    torch = pytest.importorskip("torch")
    first = build.build_fastcall()
    if first is None:
        pytest.skip("no Python headers")
    assert build.build_fastcall() == first and len(compiler) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    second = build.build_fastcall()
    assert len(compiler) == 2 and second != first and second == build.fastcall_path("0.0.1+other")


def test_the_binding_loads_the_one_for_this_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    from attention_kl_divergence_02_b200 import binding
    path = build.build_fastcall()
    if path is None:
        pytest.skip("no Python headers")
    assert binding._load_fastcall().__file__ == path
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert binding._load_fastcall() is None
