"""The build: the C library does not depend on torch, and the torch extension
follows the torch that it was built against.  In a source tree of its own.  No GPU."""
import ctypes
import os
import sys

import pytest

from exact_blocked_attention_gb300 import build as libbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "answer.cu").write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "csrc" / "torch_bind.cpp").write_text('extern "C" int bound() { return 1; }\n')
    for name, value in (("CSRC", "csrc"), ("BUILD", "_build"), ("LIB", "lib.so"), ("BIND", "bind.so")):
        monkeypatch.setattr(libbuild, name, str(tmp_path / value))
    return tmp_path


def answers(path):
    return ctypes.CDLL(path).answer() == 42


def test_the_library_is_built_without_torch(tree, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert answers(libbuild.build())
    assert not os.path.exists(libbuild.BIND)
    assert "no torch" in capfd.readouterr().err


def test_the_library_stands_where_the_extension_fails(tree):
    (tree / "csrc" / "torch_bind.cpp").write_text("#error no headers\n")
    with pytest.raises(RuntimeError, match="no headers"):
        libbuild.build()
    assert answers(libbuild.LIB)


def test_the_extension_is_rebuilt_for_another_torch(tree, monkeypatch):
    libbuild.build()
    first = os.stat(libbuild.BIND).st_ino
    libbuild.build()
    assert os.stat(libbuild.BIND).st_ino == first
    kept = os.open(libbuild.BIND, os.O_RDONLY)  # (its inode number stays taken)
    monkeypatch.setattr(libbuild, "_torch_tag", lambda: "another torch", raising=False)
    libbuild.build()
    assert os.stat(libbuild.BIND).st_ino != first
    os.close(kept)
