"""Host-side checks of blkattn_fwd_paged: its refusals come before any CUDA call.  No GPU."""
import ctypes
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn
from exact_blocked_attention_gb300 import build as libbuild

from test_abi_host import FakeTensor

I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return blkattn.load()


def args(B=2, Hq=8, Hkv=2, Tq=3, d=128, P=16, N=9, entries=4, dt=BF16):
    return dict(q=FakeTensor((B, Hq, Tq, d), dt), kp=FakeTensor((N, Hkv, P, d), dt, addr=0x100000),
                vp=FakeTensor((N, Hkv, P, d), dt, addr=0x200000), table=FakeTensor((B, entries), I32),
                sl=FakeTensor((B,), I32), qp=FakeTensor((B, Tq), I32), tree=None, window=0, scale=0.1,
                out=FakeTensor((B, Hq, Tq, d), F32, addr=0x300000), lse=FakeTensor((B, Hq, Tq), F32, addr=0x400000))


def call(lib, a):
    ref = lambda t: None if t is None else ctypes.byref(t.desc())
    return lib.blkattn_fwd_paged(ref(a["q"]), ref(a["kp"]), ref(a["vp"]), ref(a["table"]), ref(a["sl"]), ref(a["qp"]),
                                 ref(a["tree"]), a["window"], a["scale"], ref(a["out"]), ref(a["lse"]), None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), -1), (dict(kp=None), -1), (dict(vp=None), -1), (dict(table=None), -1), (dict(sl=None), -1),
    (dict(qp=None), -1), (dict(out=None), -1), (dict(lse=None), -1),
    (dict(q=FakeTensor((2, 8, 3, 128), F32)), -1),                                   # q and pools differ
    (dict(kp=FakeTensor((9, 2, 16, 128), F32, addr=0x100000)), -1),
    (dict(kp=FakeTensor((8, 2, 16, 128), BF16, addr=0x100000)), -1),                 # pools of two sizes
    (dict(kp=FakeTensor((0, 2, 16, 128), BF16), vp=FakeTensor((0, 2, 16, 128), BF16)), -1),  # no pages
    (dict(q=FakeTensor((2, 9, 3, 128), BF16), out=FakeTensor((2, 9, 3, 128), F32), lse=FakeTensor((2, 9, 3), F32)), -1),
    (dict(table=FakeTensor((3, 4), I32)), -1), (dict(table=FakeTensor((2, 4), I64)), -1),
    (dict(table=FakeTensor((2, 0), I32)), -1), (dict(table=FakeTensor((2, 4), I32, addr=None)), -1),
    (dict(table=FakeTensor((2, 4), I32, device=1)), -1),
    (dict(kp=FakeTensor((9, 2, 16, 128), BF16, strides=(4096, 2048, 128, 2), addr=0x100000)), -1),
    (dict(kp=FakeTensor((9, 2, 16, 128), BF16, strides=(4096 + 4, 2048, 128, 1), addr=0x100000)), -1),
    (dict(vp=FakeTensor((9, 2, 16, 128), BF16, addr=0x200008)), -1),                 # not 16-byte aligned
    (dict(window=-1), -1), (dict(window=1 << 31), -1),
    (dict(window=5, tree=FakeTensor((2, 3), I64)), -1), (dict(tree=FakeTensor((2, 3), I32)), -1),
    (dict(tree=FakeTensor((2, 4), I64)), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(out=FakeTensor((2, 8, 3, 128), F32, strides=(1024, 0, 128, 1), addr=0x300000)), -1),
    (dict(lse=FakeTensor((2, 8, 3), F32, strides=(0, 3, 1), addr=0x400000)), -1),
    (dict(qp=FakeTensor((2, 4), I32)), -1), (dict(sl=FakeTensor((2,), I64)), -1),
    (dict(table=FakeTensor((2, 1 << 27), I32)), -2), (dict(table=FakeTensor((2, 1 << 26), I32)), -2),
    (dict(kp=FakeTensor((9, 2, 16, 128), BF16, strides=(4096, 0, 128, 1), addr=0x100000)), -1),
    (dict(vp=FakeTensor((9, 2, 16, 128), BF16, strides=(0, 2048, 128, 1), addr=0x200000)), -1),
])
def test_refuses(lib, change, want):
    a = args()
    a.update(change)
    assert call(lib, a) == want


@pytest.mark.parametrize("kw,want", [(dict(P=4), -2), (dict(P=48), -2), (dict(P=1 << 17), -2), (dict(P=0), -1),
                                     (dict(d=96), -2), (dict(d=256), -2)])
def test_refuses_sizes(lib, kw, want):
    assert call(lib, args(**kw)) == want


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0)])
def test_no_rows_is_a_no_op(lib, kw):
    a = args(**kw)
    for n in ("q", "sl", "qp", "out", "lse"):
        a[n].addr = None
    if kw.get("B") == 0:
        a["table"].addr = None
    assert call(lib, a) == 0
