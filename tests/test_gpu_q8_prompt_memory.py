"""Memory of prompts over the 8-bit cache: what the library's copy of the pages
takes, and calls whose copy finds no memory.  Each runs in a process of its own,
whose device memory pool is one that the test can limit and look into."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HEAD = """
import ctypes, sys
sys.path[:0] = [%r, %r]
import torch
from exact_blocked_attention_gb300 import blkattn
from test_gpu_paged_q8 import BF16, F32, I32, call, check, make

class Props(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("handles", ctypes.c_int), ("where", ctypes.c_int), ("id", ctypes.c_int),
                ("security", ctypes.c_void_p), ("most", ctypes.c_size_t), ("usage", ctypes.c_ushort),
                ("reserved", ctypes.c_ubyte * 54)]

cu = ctypes.CDLL("libcuda.so.1")
torch.zeros(1, device="cuda")
pool = ctypes.c_void_p()
props = Props(type=1, where=1, id=0, most=MOST)
assert cu.cuMemPoolCreate(ctypes.byref(pool), ctypes.byref(props)) == 0
assert cu.cuDeviceSetMemPool(0, pool) == 0

def used():  # bytes of the pool that are taken
    torch.cuda.synchronize()
    n = ctypes.c_uint64()
    assert cu.cuMemPoolGetAttribute(pool, 7, ctypes.byref(n)) == 0
    return n.value

MIB = 1 << 20
"""


def run(most, body):
    here = os.path.dirname(os.path.abspath(__file__))
    text = HEAD.replace("MOST", str(most)) % (here, os.path.dirname(here)) + body + "\nprint('done')\n"
    p = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("done"), p.stdout[-500:] + p.stderr[-3000:]


def test_a_copy_that_finds_no_memory():
    """In a pool of 96 MiB: four sequences of 24 MiB each (and their tables), by slices; one of 128 MiB, heads apart; a
    head of 256 MiB, without a copy."""
    run(96 << 20, """
for a in (make(4, 2, 1, 64, 128, 64, 16, [300, 64, 1000, 2000], entries=768, heads_first=True),
          make(1, 8, 4, 100, 64, 64, 16, [1500], entries=2048, heads_first=True),
          make(2, 2, 1, 64, 128, 64, 16, [900, 100], entries=8192, heads_first=True)):
    for out in (BF16, F32):
        want = call(a, out)
        check(a, want, out)
        assert used() <= 96 * MIB
        g = torch.cuda.CUDAGraph()  # captured, the call does the same
        with torch.cuda.graph(g):
            got = call(a, out)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
""")


def test_captured_without_a_call_before():
    run(0, """
a = make(1, 2, 1, 64, 128, 64, 16, [300], entries=768, heads_first=True)
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        call(a, BF16)
except blkattn.BlkattnError as e:
    assert "-5" in str(e), e
else:
    raise AssertionError("grown under capture")
""")


def test_what_growing_copies_hold():
    """Sequences of 0.3 to 9 GiB, one after another: 2 GiB are held, and less than that of outgrown buffers."""
    run(0, """
for rows in (150, 350, 700, 1300, 1600, 4600):
    a = make(1, 8, 4, 64, 128, 64, 16, [500], entries=rows * 1024 // 64, heads_first=True, seed=rows)
    check(a, call(a, BF16), BF16)
assert 2048 * MIB <= used() < (4096 + 64) * MIB, used() / MIB
a = make(3, 8, 4, 64, 128, 64, 16, [500, 100, 300], entries=12288, heads_first=True)
check(a, call(a, BF16), BF16)
assert used() < (4096 + 64) * MIB, used() / MIB
""")


def test_a_long_single_head():
    """A head whose copy would pass 2 GiB: the pages are read as they are."""
    run(0, """
a = make(1, 2, 1, 64, 128, 256, 16, [3000], entries=5 * 4096 + 7, heads_first=True)
check(a, call(a, BF16), BF16)
assert used() < 64 * MIB, used() / MIB
""")


def test_random_prompts_in_slices():
    """Problems of every kind whose copies go by sequences, by heads or not at all, the workspace beside them in
    what is left."""
    run(160 << 20, """
import random
r = random.Random(5)
for seed in range(40):
    d, P = r.choice([64, 128]), r.choice([16, 64, 256])
    S = min(P, r.choice([1, 4, 16, 64]))
    Hkv, T, B = r.choice([1, 2, 3, 5, 8]), r.choice([64, 65, 100, 300]), r.choice([1, 2, 3, 5])
    Hq = Hkv * r.choice([1, 2, 3])
    lens = [r.randint(T, T + r.choice([10, 600, 2500])) for _ in range(B)]
    wide = r.choice([1, 8, 60, 200]) * 1024 * 128 // (d * P)
    a = make(B, Hq, Hkv, T, d, P, S, lens, seed=seed, heads_first=r.random() < 0.5, rows_major=r.random() < 0.3,
             entries=max(wide, 2800 // P + 2))
    mode = r.choice(["causal", "window", "holes"])
    if mode == "window":
        a["window"] = r.choice([1, 50, 700])
    if mode == "holes":
        a["table"][r.randrange(B), r.randrange(max(1, min(lens) // P))] = -1
        a["pos"][0, r.randrange(T)] = -1
    out = r.choice([BF16, F32])
    check(a, call(a, out), out)
    assert used() <= 160 * MIB
""")


def test_a_workspace_that_finds_no_memory():
    """Beside a copy: the copy gives its memory back, and a captured call does as this one did.  Alone: an error of that
    call only."""
    for most in (64, 96):
        run(most << 20, """
big = make(192, 24, 8, 48, 128, 64, 16, [48] * 192)
small = make(2, 8, 2, 1, 128, 16, 16, [300, 400])
a = make(2, 32, 1, 200, 128, 64, 16, [4000, 900], entries=1400, heads_first=True)  # 44 MiB of pages each, 17 of parts
want = call(a, BF16)
check(a, want, BF16)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call(a, BF16)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
try:
    call(big, F32)
except blkattn.BlkattnError as e:
    assert "memory" in str(e), e
else:
    raise AssertionError("a workspace of more than the pool")
check(small, call(small, BF16), BF16)
""")
