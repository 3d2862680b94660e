"""Growth of the library's scratch where memory is short: what fits is not
refused because twice the old size does not.  The rule alone, compiled for the
host with a fake allocator.  No GPU."""
import ctypes
import os
import subprocess

import pytest

from exact_blocked_attention_gb300 import build as libbuild

SHIM = """
#include "scratch.h"
enum { kNoMemory = 2, kOther = 7 };
extern "C" int grow(size_t have, size_t need, size_t room, int broken, size_t* got, int* asked) {
  *asked = 0;
  return blkattn::grow_scratch(
      have, need, [&](size_t n) { ++*asked; return broken ? kOther : n <= room ? 0 : kNoMemory; },
      [](int e) { return e == kNoMemory; }, got);
}
"""


@pytest.fixture(scope="module")
def grow(tmp_path_factory):
    at = tmp_path_factory.mktemp("scratch")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-I", libbuild.CSRC, str(at / "shim.cpp"), "-o",
                    str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(os.path.join(at, "shim.so"))
    lib.grow.argtypes = [ctypes.c_size_t] * 3 + [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]

    def call(have, need, room, broken=0):
        got, asked = ctypes.c_size_t(), ctypes.c_int()
        st = lib.grow(have, need, room, broken, ctypes.byref(got), ctypes.byref(asked))
        return st, got.value, asked.value

    return call


@pytest.mark.parametrize("have,need,room,want", [
    (0, 100, 1000, (0, 100, 1)), (100, 150, 1000, (0, 200, 1)), (100, 200, 1000, (0, 200, 1)),
    (100, 500, 1000, (0, 500, 1)),
    (600, 700, 1000, (0, 700, 2)),   # twice does not fit, the need does
    (600, 1000, 1000, (0, 1000, 2)),
    (600, 1001, 1000, (2, 1001, 2)), (100, 2000, 1000, (2, 2000, 1))])
def test_growth(grow, have, need, room, want):
    assert grow(have, need, room) == want


def test_another_error_is_not_asked_again(grow):
    assert grow(600, 700, 5000, broken=1) == (7, 1200, 1)
