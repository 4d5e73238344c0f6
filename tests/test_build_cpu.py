"""The short way's module (csrc/fastcall.cpp) is optional: it belongs to one
torch and one Python, and neither the build nor the calls need it."""
import os
import stat

import pytest
import torch

import cross_layer_top_full_b200 as ic
from cross_layer_top_full_b200 import build as icbuild


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """A stand-in for the compiler and a place for what it makes: compiler(script body)."""
    monkeypatch.setattr(icbuild, "PKG", str(tmp_path))
    log = tmp_path / "calls"

    def make(body):
        exe = tmp_path / "compiler"
        exe.write_text("#!/bin/sh\necho call >> %s\n%s\n" % (log, body))
        exe.chmod(exe.stat().st_mode | stat.S_IEXEC)
        monkeypatch.setattr(icbuild.shutil, "which", lambda name: str(exe))
        return lambda: len(log.read_text().split()) if log.exists() else 0

    return make


WRITES = 'while [ "$1" != "-o" ]; do shift; done; echo made > "$2"'


def test_the_module_names_its_torch_and_python(monkeypatch):
    path = icbuild.fast_path()
    assert torch.__version__ in path and "cpython" in path
    monkeypatch.setattr(torch, "__version__", "9.9")
    assert icbuild.fast_path() != path


def test_another_torch_gets_a_module_of_its_own(compiler, monkeypatch):
    calls = compiler(WRITES)
    icbuild._build_fastcall(False)
    first = icbuild.fast_path()
    assert os.path.exists(first) and calls() == 1
    icbuild._build_fastcall(False)                       # it is there
    assert calls() == 1
    monkeypatch.setattr(torch, "__version__", "9.9")
    icbuild._build_fastcall(False)
    assert calls() == 2 and os.path.exists(icbuild.fast_path()) and not os.path.exists(first)


@pytest.mark.parametrize("old", [False, True])
def test_a_failed_compile_is_said_and_leaves_no_module(old, compiler, capfd):
    compiler("echo no Python.h >&2; exit 1")
    fast = icbuild.fast_path()
    if old:                                              # made of older sources
        open(fast, "w").close()
        os.utime(fast, (1, 1))
    icbuild._build_fastcall(False)
    err = capfd.readouterr().err
    assert "no Python.h" in err and "the long way" in err
    assert not os.path.exists(fast)


def test_no_compiler_is_no_error(compiler, monkeypatch, capfd):
    compiler("")
    monkeypatch.setattr(icbuild.shutil, "which", lambda name: "/nonexistent/compiler")
    icbuild._build_fastcall(False)
    assert "the long way" in capfd.readouterr().err


def test_the_calls_go_the_long_way_without_the_module(monkeypatch, tmp_path):
    monkeypatch.setattr(icbuild, "PKG", str(tmp_path))
    assert ic._Torch().fast is None
    monkeypatch.setattr(torch, "__version__", "9.9")     # a module of another torch is not loaded
    (tmp_path / "_fastcall.so").write_text("")
    assert ic._Torch().fast is None
    open(icbuild.fast_path(), "w").close()               # nor one that is broken
    assert ic._Torch().fast is None
