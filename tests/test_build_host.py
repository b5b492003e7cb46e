"""build_host() (CPU): when wb_host.so is compiled, kept and removed.  The compiler is a stand-in that writes a file, or fails."""
import os
import subprocess

import pytest

from whisper_encoder_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree and build folder of its own, and the list of compilations that were asked for; tree.works = False: they fail."""
    class Tree:
        works, calls = True, []

        def compile(self, cmd, **kw):
            self.calls.append(cmd)
            if not self.works:
                return subprocess.CompletedProcess(cmd, 1, "", "no Python.h")
            with open(cmd[cmd.index("-o") + 1], "w") as fh:
                fh.write(f"library {len(self.calls)}")
            return subprocess.CompletedProcess(cmd, 0, "", "")

    t = Tree()
    t.calls = []
    csrc, include, out = tmp_path / "csrc", tmp_path / "include", tmp_path / "_build"
    csrc.mkdir()
    include.mkdir()
    t.source = csrc / build.HOST_SOURCE
    t.source.write_text("one")
    (include / "wb.h").write_text("header")
    t.header = include / "wb.h"
    t.lib = out / "wb_host.so"
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(out))
    monkeypatch.setattr(build, "LIB_HOST", str(t.lib))
    monkeypatch.setattr(build.subprocess, "run", t.compile)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return t


def _no_nvcc():
    raise RuntimeError("nvcc not found")


def test_compiled_once(tree):
    assert build.build_host() == str(tree.lib) and build.build_host() == str(tree.lib)
    assert len(tree.calls) == 1 and tree.lib.read_text() == "library 1"
    assert build.build_host(force=True) == str(tree.lib) and len(tree.calls) == 2


@pytest.mark.parametrize("what", ["source", "header", "torch"])
def test_compiled_again_where_something_it_depends_on_changed(tree, monkeypatch, what):
    build.build_host()
    if what == "torch":
        monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0")
    else:
        getattr(tree, what).write_text("two")
    assert build.build_host() == str(tree.lib) and len(tree.calls) == 2


def test_a_current_library_needs_no_compiler(tree, monkeypatch):
    build.build_host()
    monkeypatch.setattr(build, "_nvcc", _no_nvcc)
    assert build.build_host() == str(tree.lib) and tree.lib.exists()
    monkeypatch.setattr(build, "_nvcc", lambda: "/opt/other/bin/nvcc")
    monkeypatch.setenv("CXX", "/opt/other/bin/g++")
    assert build.build_host() == str(tree.lib) and len(tree.calls) == 1


def test_a_forced_compilation_that_fails_keeps_a_current_library(tree, capfd):
    build.build_host()
    tree.works = False
    assert build.build_host(force=True) is None and tree.lib.exists()
    assert "no Python.h" in capfd.readouterr().err


@pytest.mark.parametrize("how", ["compiler fails", "no nvcc"])
@pytest.mark.parametrize("stamped", [True, False])
def test_a_library_of_another_source_does_not_stay(tree, monkeypatch, capfd, how, stamped):
    build.build_host()
    if not stamped:
        os.remove(tree.lib.parent / "host_digest.txt")
    tree.source.write_text("two")
    tree.works = False
    if how == "no nvcc":
        monkeypatch.setattr(build, "_nvcc", _no_nvcc)
    assert build.build_host() is None and not tree.lib.exists()
    assert "wb_host.so is not built" in capfd.readouterr().err
    tree.works = True
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    assert build.build_host() == str(tree.lib) and tree.lib.exists()


def test_an_interpreter_that_cannot_tell_removes_nothing(tree, monkeypatch, capfd):
    def missing(name):
        raise build.importlib.metadata.PackageNotFoundError(name)

    build.build_host()
    monkeypatch.setattr(build.importlib.metadata, "version", missing)
    assert build.build_host() is None and tree.lib.exists() and len(tree.calls) == 1
    assert "wb_host.so is not built" in capfd.readouterr().err
