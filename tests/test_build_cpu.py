"""CPU checks of the build around the compilers: what happens without one, and what is built again."""

import os
import subprocess
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
from moe_lora_virtual_gb300 import build  # noqa: E402


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Stand-ins: every command writes its output file; `missing` is not on the path."""
    seen = SimpleNamespace(ran=[], missing=None, failing=None, waited=0)
    for name in ("LIB_PATH", "CHECKED_LIB_PATH", "NATIVE_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "NATIVE_STAMP", build.NATIVE_PATH + ".stamp")
    monkeypatch.setattr(build, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")

    class Popen:
        def __init__(self, cmd, **_):
            self.name = os.path.basename(cmd[0])
            if self.name == seen.missing:
                raise FileNotFoundError(2, "No such file or directory", self.name)
            seen.ran.append(self.name)
            self.returncode = int(self.name == seen.failing)
            if not self.returncode:
                open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            seen.waited += 1
            return "what the compiler says", None

    monkeypatch.setattr(subprocess, "Popen", Popen)
    return seen


def test_builds_once(compilers):
    build.build_all()
    assert sorted(compilers.ran) == ["g++", "nvcc", "nvcc"] and build.native_current()
    build.build_all()
    assert len(compilers.ran) == 3


@pytest.mark.parametrize("kind", ["missing", "failing"])
def test_without_native_calls_the_libraries_are_built(compilers, kind):
    setattr(compilers, kind, "g++")
    with pytest.warns(UserWarning, match="_block_native.so was not built"):
        paths = build.build_all()
    assert all(os.path.exists(p) for p in paths) and not os.path.exists(build.NATIVE_PATH)
    assert compilers.waited == len(compilers.ran) and not build.native_current()
    setattr(compilers, kind, None)
    compilers.ran.clear()
    build.build_all()
    assert compilers.ran == ["g++"] and build.native_current()


def test_without_pytorch_the_libraries_are_built(compilers, monkeypatch):
    def command(out):
        raise ImportError("no torch")

    monkeypatch.setattr(build, "_native_command", command)
    with pytest.warns(UserWarning, match="no torch"):
        paths = build.build_all()
    assert all(os.path.exists(p) for p in paths)


def test_a_library_that_does_not_build_is_an_error(compilers):
    compilers.failing = "nvcc"
    with pytest.raises(RuntimeError, match="what the compiler says"):
        build.build_all()
    assert compilers.waited == 3


@pytest.mark.parametrize("what", ["torch", "python", "none"])
def test_native_calls_for_another_pytorch_are_built_again(compilers, monkeypatch, what):
    build.build_all()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "2.99.0")
    elif what == "python":
        monkeypatch.setattr(build.sys, "version", "3.99")
    else:
        os.remove(build.NATIVE_STAMP)
    assert not build.native_current()
    compilers.ran.clear()
    build.build_all()
    assert compilers.ran == ["g++"] and build.native_current()
