"""Slices of an 8-bit cache's copy for prompts, and the buffer that holds them:
the rule alone, compiled for the host with a fake allocator.  No GPU."""
import ctypes
import os
import random
import subprocess

import pytest

from exact_blocked_attention_gb300 import build as libbuild

SHIM = """
#include "scratch.h"
enum { kNoMemory = 2, kOther = 7 };
extern "C" void fit(int64_t B, int64_t H, int64_t seq, int64_t head, int64_t most, int64_t* have, int64_t* room, int broken,
                    int64_t* out, int64_t* asked) {
  int failed = -1, n = 0;
  const blkattn::Slice s = blkattn::fit_slices(
      B, H, seq, head, most, have,
      [&](int64_t b) {
        if (n < 64) asked[n++] = b;
        if (broken) return (int)kOther;
        if (b > *room) return (int)kNoMemory;
        *room -= b;
        return 0;
      },
      [](int e) { return e == kNoMemory; }, &failed);
  out[0] = s.seqs; out[1] = s.heads; out[2] = failed; out[3] = n;
}
"""


@pytest.fixture(scope="module")
def fit(tmp_path_factory):
    at = tmp_path_factory.mktemp("slices")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", libbuild.CSRC, str(at / "shim.cpp"),
                    "-o", str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(os.path.join(at, "shim.so"))
    I, P = ctypes.c_int64, ctypes.c_void_p
    lib.fit.argtypes = [I, I, I, I, I, P, P, ctypes.c_int, P, P]

    def call(B, H, seq, head, most, have=0, room=1 << 60, broken=0):
        h, r, out, asked = I(have), I(room), (I * 4)(), (I * 64)()
        lib.fit(B, H, seq, head, most, ctypes.byref(h), ctypes.byref(r), broken, out, asked)
        return (out[0], out[1]), out[2], list(asked[:out[3]]), h.value, r.value

    return call


@pytest.mark.parametrize("B,H,seq,head,want,asked", [
    (3, 2, 0, 100, (3, 2), [1024]), (1, 1, 1, 127, (1, 1), [128]), (1, 1, 1, 128, (1, 1), [256]),
    (8, 4, 10, 60, (4, 4), [1024]),              # 250 a sequence: four of them
    (8, 8, 24, 250, (1, 4), [1024]),             # a sequence is 2024: half of its heads
    (2, 9, 24, 250, (1, 3), [1024]),             # (nine in three times three, not four, four and one)
    (2, 9, 24, 1000, (1, 1), [1024]), (2, 9, 25, 1000, (0, 0), []), (0, 9, 25, 10, (0, 0), []), (3, 0, 25, 10, (0, 0), [])])
def test_what_a_slice_takes(fit, B, H, seq, head, want, asked):
    got, failed, n, have, _ = fit(B, H, seq, head, 1024)
    assert (got, failed, n) == (want, 0, asked) and have == sum(asked)


def test_a_buffer_that_is_large_enough_stays(fit):
    assert fit(4, 4, 10, 60, 1024, have=1000)[:4] == ((4, 4), 0, [], 1000)


@pytest.mark.parametrize("room,have,want,asked,now", [
    (1000, 0, (4, 4), [1024, 1000], 1000),               # the rounded size finds none, the need does
    (999, 0, (2, 4), [1024, 1000, 512], 512),            # half as many
    (500, 0, (2, 4), [1024, 1000, 512, 500], 500),
    (499, 256, (1, 4), [1024, 1000, 512, 500], 256),     # one, in what is there
    (100, 0, (1, 1), [1024, 1000, 512, 500, 256, 250, 256, 130, 128, 70], 70),
    (69, 0, (0, 0), [1024, 1000, 512, 500, 256, 250, 256, 130, 128, 70], 0)])
def test_short_memory(fit, room, have, want, asked, now):
    got, failed, n, held, _ = fit(4, 4, 10, 60, 1024, have=have, room=room)
    assert (got, failed, n, held) == (want, 0, asked, now)


def test_another_error_ends_it(fit):
    assert fit(4, 4, 10, 60, 1024, broken=1)[:3] == ((0, 0), 7, [1024])


@pytest.mark.parametrize("seed", range(50))
def test_what_is_held_stays_bounded(fit, seed):
    """With memory enough, all buffers ever asked for together stay below twice the most."""
    r = random.Random(seed)
    have, held = 0, 0
    for _ in range(30):
        B, H, seq, head = r.randint(1, 50), r.randint(1, 16), r.randint(1, 1000), r.randint(1, 1 << r.randint(1, 21))
        (seqs, heads), failed, n, have, _ = fit(B, H, seq, head, 1 << 20, have=have)
        held += sum(n)
        assert failed == 0 and held < 2 << 20 and have <= 1 << 20
        if seqs:
            assert seqs <= B and heads <= H and (seqs == 1 or heads == H) and seqs * (seq + heads * head) <= have
        else:
            assert seq + head > 1 << 20


def test_the_same_size_is_not_asked_twice(fit):
    assert fit(1, 1, 0, 512, 1024, room=511)[:3] == ((0, 0), 0, [512])
