"""What is built when, with compilers that only write their output files: the
library stands by itself, the draft calls' binding needs torch as well."""
from __future__ import annotations

import os
import sys

import pytest

from affine_bit_group_gb300 import _build

COMPILER = """#!/bin/sh
echo "$@" >> {log}
case "$*" in *"$FAIL"*) echo "no such header"; exit 1;; esac
while [ $# -gt 0 ]; do
    if [ "$1" = -o ]; then echo x > "$2"; fi
    shift
done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into tmp_path; returns a function that gives the compilers' calls since it was last asked."""
    log = tmp_path / "log"
    exe = tmp_path / "compiler"
    exe.write_text(COMPILER.format(log=log))
    exe.chmod(0o755)
    for name, value in (("NVCC", str(exe)), ("CXX", str(exe)), ("OBJ", str(tmp_path / "obj")),
                        ("LIB", str(tmp_path / "libabg.so")), ("MARSHAL", str(tmp_path / "_marshal.so"))):
        monkeypatch.setattr(_build, name, value, raising=name != "CXX")
    monkeypatch.setenv("FAIL", "nothing fails")

    def calls():
        text = log.read_text() if log.exists() else ""
        log.write_text("")
        return text

    return calls


def test_library_is_built_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert _build.stale()
    _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.MARSHAL)
    assert "marshal" not in tree() and not _build.stale() and not _build.marshal_stale()
    _build.build()
    assert tree() == ""


def test_library_is_linked_where_the_binding_does_not_compile(tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("FAIL", "marshal.cpp")
    with pytest.raises(RuntimeError, match="marshal.cpp:\nno such header"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.MARSHAL)
    assert not _build.stale() and _build.marshal_stale()


def test_a_missing_binding_does_not_rebuild_the_library(tree):
    pytest.importorskip("torch")
    _build.build()
    assert ".cu " in tree() and os.path.exists(_build.MARSHAL)
    os.remove(_build.MARSHAL)
    assert not _build.stale()
    _build.build()
    calls = tree()
    assert "marshal.cpp" in calls and ".cu " not in calls and os.path.exists(_build.MARSHAL)
    _build.build(marshal=False)
    assert tree() == ""


def test_library_errors_are_told(tree, monkeypatch):
    monkeypatch.setenv("FAIL", "vec.cu")
    with pytest.raises(RuntimeError, match="vec.cu:\nno such header"):
        _build.build()
    assert not os.path.exists(_build.LIB) and not os.path.exists(_build.MARSHAL)


def test_binding_is_rebuilt_for_another_torch(tree, monkeypatch, tmp_path):
    """Whatever the files' times: the module is compiled against torch's headers."""
    pytest.importorskip("torch")
    _build.build()
    tree()
    assert not _build.marshal_stale()
    root = tmp_path / "torch"
    root.mkdir()
    (root / "version.py").write_text("__version__ = '2.99'\n")
    monkeypatch.setattr(_build, "_torch_root", lambda: str(root))
    assert _build.marshal_stale() and not _build.stale()
    _build.build()
    assert str(root) in tree() and not _build.marshal_stale()
    (root / "version.py").write_text("__version__ = '3.0'\n")
    assert _build.marshal_stale()
