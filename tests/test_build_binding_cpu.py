"""The build where the native marshalling module cannot be compiled (no C++20
compiler, no headers of torch): the library is built, with a warning, and no stale
module stays behind.  The compilers are stand-ins here."""
import pathlib
import types
import warnings

import pytest

from vocab_wide_token_gb300 import build


def _toolchain(monkeypatch, tmp_path, gxx):
    def run(cmd, **_):
        if cmd[0] == "g++":
            return gxx(cmd)
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_text("linked")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpstat.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "nvcc", lambda: "/opt/cuda/bin/nvcc")
    monkeypatch.setattr(build, "_compile", lambda src, *_: src)
    monkeypatch.setattr(build.subprocess, "run", run)


def _fails(cmd):
    return types.SimpleNamespace(returncode=1, stdout="", stderr="unrecognized option -std=c++20")


def _is_missing(cmd):
    raise FileNotFoundError(2, "No such file or directory", "g++")


@pytest.mark.parametrize("gxx", [_fails, _is_missing])
def test_the_library_is_built_without_the_module(monkeypatch, tmp_path, gxx):
    _toolchain(monkeypatch, tmp_path, gxx)
    (tmp_path / "_binding.so").write_text("of an earlier build")
    with pytest.warns(RuntimeWarning, match="_binding"):
        assert build.build() == build.LIB
    assert (tmp_path / "libpstat.so").read_text() == "linked"
    assert not (tmp_path / "_binding.so").exists()


def test_both_are_built(monkeypatch, tmp_path):
    def gxx(cmd):
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_text("module")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    _toolchain(monkeypatch, tmp_path, gxx)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build()
    assert (tmp_path / "_binding.so").read_text() == "module"


def test_a_kernel_that_does_not_compile_still_fails(monkeypatch, tmp_path):
    _toolchain(monkeypatch, tmp_path, _fails)

    def compile_fails(src, *_):
        raise RuntimeError("nvcc failed on " + src)

    monkeypatch.setattr(build, "_compile", compile_fails)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    assert not (tmp_path / "libpstat.so").exists()
