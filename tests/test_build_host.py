"""The binding's CPython extension is optional: a build without Python's headers or without a working C
compiler still gives the library, and leaves no extension behind that was built from an older source."""
import os
import subprocess

import pytest

from bit_w4a4_quantized_group_b200 import build as BUILD


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """An up-to-date library, an extension built before its source last changed, and nvcc out of reach."""
    lib, calls, csrc = tmp_path / "libsvdq.so", tmp_path / "svdq_call.so", tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "svdq_call.c").write_text("int x;\n")
    (csrc / "a.cu").write_text("")
    calls.write_text("old")
    lib.write_text("library")
    os.utime(calls, (1, 1))
    monkeypatch.setattr(BUILD, "CALLS", str(calls))
    monkeypatch.setattr(BUILD, "LIB", str(lib))
    monkeypatch.setattr(BUILD, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(BUILD, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(BUILD, "CSRC", str(csrc))
    monkeypatch.setattr(BUILD, "_compile", lambda *a: "x.o")
    return lib, calls


def _tools(monkeypatch, gcc):
    def run(cmd, **kw):
        if cmd[0] == "gcc":
            return gcc(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("linked")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(BUILD.subprocess, "run", run)


def _fails(cmd):
    return subprocess.CompletedProcess(cmd, 1, "", "internal compiler error")


def _missing(cmd):
    raise FileNotFoundError("gcc")


@pytest.mark.parametrize("gcc", [_fails, _missing])
@pytest.mark.parametrize("stale_library", [False, True])
def test_a_compiler_that_fails_costs_the_extension_alone(sandbox, monkeypatch, capsys, gcc, stale_library):
    lib, calls = sandbox
    if stale_library:
        os.utime(lib, (1, 1))
    monkeypatch.setattr(BUILD, "_python_include", lambda: "/include")
    _tools(monkeypatch, gcc)
    assert BUILD.build() == str(lib)
    assert not calls.exists() and "ctypes alone" in capsys.readouterr().err
    assert lib.read_text() == ("linked" if stale_library else "library")
    assert BUILD.build() == str(lib) and lib.read_text() == ("linked" if stale_library else "library")


def test_without_headers_an_old_extension_goes(sandbox, monkeypatch):
    lib, calls = sandbox
    monkeypatch.setattr(BUILD, "_python_include", lambda: "")
    _tools(monkeypatch, _missing)
    assert BUILD.build() == str(lib) and not calls.exists()


def test_an_extension_newer_than_its_source_stays(sandbox, monkeypatch):
    lib, calls = sandbox
    os.utime(calls, None)
    monkeypatch.setattr(BUILD, "_python_include", lambda: "")
    _tools(monkeypatch, _missing)
    assert BUILD.build() == str(lib) and calls.read_text() == "old"


def test_a_working_compiler_replaces_it(sandbox, monkeypatch):
    lib, calls = sandbox

    def gcc(cmd):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(BUILD, "_python_include", lambda: "/include")
    _tools(monkeypatch, gcc)
    assert BUILD.build() == str(lib) and calls.read_text() == "new"
