"""The build of the compiled calls beside the library (no GPU, no compiler): when _front.so is out of date, that a front
which cannot be built leaves the library built, and what loading one that does not fit says."""
import os
import time

import pytest

import kernelized_causal_attention_gb300 as la
from kernelized_causal_attention_gb300 import _build as b


def _tree(tmp_path, monkeypatch):
    """A source tree with everything built 100 s after its last change, but for what the test changes."""
    csrc, lib = tmp_path / "csrc", tmp_path / "_lib"
    csrc.mkdir()
    lib.mkdir()
    for d, n in ((csrc, "a.cu"), (csrc, "k.cuh"), (csrc, "front.cpp"), (tmp_path, "linattn.h"), (tmp_path, "_build.py")):
        (d / n).write_text("// text\n")
        os.utime(d / n, (time.time() - 100,) * 2)
    for n, v in (("CSRC", csrc), ("LIBDIR", lib), ("LIB", lib / "liblinattn.so"), ("FRONT", lib / "_front.so"), ("INCLUDE", tmp_path),
                 ("MANIFEST", lib / "sources.txt"), ("FRONT_MANIFEST", lib / "front.txt"), ("__file__", tmp_path / "_build.py")):
        monkeypatch.setattr(b, n, str(v))
    (lib / "liblinattn.so").write_bytes(b"\0")
    (lib / "_front.so").write_bytes(b"\0")
    (lib / "sources.txt").write_text(b._manifest())
    (lib / "front.txt").write_text(b.front_manifest())
    return csrc, lib


def test_both_are_up_to_date(tmp_path, monkeypatch):
    _tree(tmp_path, monkeypatch)
    assert b.up_to_date() and b.front_up_to_date()
    monkeypatch.setattr(b, "_run", lambda *a: pytest.fail("nothing is to be run"))
    assert b.build() == b.LIB


@pytest.mark.parametrize("name", ["_front.so", "front.txt"])
def test_a_missing_front(tmp_path, monkeypatch, name):
    _, lib = _tree(tmp_path, monkeypatch)
    (lib / name).unlink()
    assert b.up_to_date() and not b.front_up_to_date()


def test_a_newer_front_source(tmp_path, monkeypatch):
    csrc, lib = _tree(tmp_path, monkeypatch)
    os.utime(csrc / "front.cpp", (time.time() + 100,) * 2)
    assert b.up_to_date() and not b.front_up_to_date()


def test_a_newer_header_or_recipe(tmp_path, monkeypatch):
    _tree(tmp_path, monkeypatch)
    for n in ("linattn.h", "_build.py"):
        os.utime(tmp_path / n, (time.time() + 100,) * 2)
        assert not b.up_to_date() and not b.front_up_to_date()
        os.utime(tmp_path / n, (time.time() - 100,) * 2)
    assert b.up_to_date() and b.front_up_to_date()


def test_a_newer_unit_leaves_the_front(tmp_path, monkeypatch):
    csrc, _ = _tree(tmp_path, monkeypatch)
    os.utime(csrc / "k.cuh", (time.time() + 100,) * 2)
    assert not b.up_to_date() and b.front_up_to_date()


@pytest.mark.parametrize("said", ["torch 2.0.0\npython 3.12", "torch 2.0.0"])
def test_another_torch_or_python(tmp_path, monkeypatch, said):
    _, lib = _tree(tmp_path, monkeypatch)
    (lib / "front.txt").write_text(said)
    assert b.up_to_date() and not b.front_up_to_date()
    monkeypatch.setattr(la, "_front", None)
    with pytest.raises(RuntimeError, match="torch 2.0.0.*this is torch"):
        la._load_front()


def test_a_front_that_is_not_there(tmp_path, monkeypatch):
    _, lib = _tree(tmp_path, monkeypatch)
    (lib / "_front.so").unlink()
    monkeypatch.setattr(la, "_front", None)
    with pytest.raises(RuntimeError, match="not built"):
        la._load_front()


def _compilers(monkeypatch, ran, front_fails):
    """The compilers as a function that writes the file they are asked for."""
    def run(cmd, what):
        ran.append(what)
        if front_fails and what == "front.cpp":
            raise RuntimeError("g++ failed on front.cpp:\nPython.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)
        return ""
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "/none/bin/nvcc")


def test_a_front_that_cannot_be_built_leaves_the_library(tmp_path, monkeypatch):
    _, lib = _tree(tmp_path, monkeypatch)
    ran = []
    _compilers(monkeypatch, ran, True)
    for n in ("liblinattn.so", "_front.so", "sources.txt", "front.txt"):
        (lib / n).unlink()
    with pytest.raises(RuntimeError, match="(?s)liblinattn.so is built; _front.so.*Python.h"):
        b.build()
    assert b.up_to_date() and not b.front_up_to_date() and not (lib / "_front.so").exists()
    assert (lib / "liblinattn.so").read_text() == "the library"
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()                                  # asked again: only the front is tried
    assert ran.count("the library") == 1
    _compilers(monkeypatch, ran, False)
    assert b.build() == b.LIB and b.front_up_to_date() and ran.count("the library") == 1


def test_the_library_alone(tmp_path, monkeypatch):
    _, lib = _tree(tmp_path, monkeypatch)
    ran = []
    _compilers(monkeypatch, ran, True)
    assert b.library(force=True) == b.LIB
    assert "front.cpp" not in ran and "_front.so" not in ran and b.up_to_date()


@pytest.mark.parametrize("alone", [False, True])
def test_a_front_of_another_header_is_not_loaded(tmp_path, monkeypatch, alone):
    """The ABI's header changes and only the library can be built, or is asked for: the older _front.so would call it by the
    header before."""
    _, lib = _tree(tmp_path, monkeypatch)
    ran = []
    _compilers(monkeypatch, ran, True)
    for n in ("liblinattn.so", "_front.so"):
        os.utime(lib / n, (time.time() - 50,) * 2)
    os.utime(tmp_path / "linattn.h", (time.time() - 20,) * 2)
    if alone:
        b.library()
    else:
        with pytest.raises(RuntimeError, match="Python.h"):
            b.build()
    assert b.up_to_date() and not b.front_up_to_date()
    monkeypatch.setattr(la, "_front", None)
    with pytest.raises(RuntimeError, match="not built"):
        la._load_front()


def test_everything_again(tmp_path, monkeypatch):
    _, lib = _tree(tmp_path, monkeypatch)
    ran = []
    _compilers(monkeypatch, ran, False)
    b.build(force=True)
    assert sorted(ran) == sorted([str(tmp_path / "csrc" / "a.cu"), "front.cpp", "the library", "_front.so"])
    assert b.up_to_date() and b.front_up_to_date()


def test_a_manifest_is_whole_or_not_there(tmp_path, monkeypatch):
    """What a process that loads meanwhile reads: the text before until the text after is complete."""
    _, lib = _tree(tmp_path, monkeypatch)
    real, seen = os.replace, []

    def replace(a, c):
        seen.append((lib / "front.txt").read_text())
        real(a, c)
    monkeypatch.setattr(os, "replace", replace)
    b._say(b.FRONT_MANIFEST, "torch 9\npython 9")
    assert seen == [b.front_manifest()] and (lib / "front.txt").read_text() == "torch 9\npython 9"
    assert [f.name for f in lib.iterdir() if "tmp" in f.name] == []
