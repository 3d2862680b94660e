"""Host-side checks of the rotary and paged-append operators: the angle and
phase tables, and the refusals, which come before any CUDA call.  No GPU."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn
from exact_blocked_attention_gb300 import build as libbuild

from test_abi_host import FakeTensor

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return blkattn.load()


def ref(t):
    return None if t is None else ctypes.byref(t.desc())


# ------------------------------------------------------------------ tables
def test_phases_are_the_exact_turn_fractions():
    # the header's bound: two units of 2^-64 turns
    angles = [10000.0 ** (-2 * i / 128) for i in range(64)] + [8.0, -8.0, -0.3, 0.0, 1e-30, 5e-324, 2.0 ** -60]
    for a, f in zip(angles, blkattn.rope_phases(angles, device="cpu").tolist()):
        d = (f - Fraction(a) * 2 ** 64 / TWO_PI) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= 2, a


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 8.5])
def test_phases_refuse(bad):
    with pytest.raises(ValueError):
        blkattn.rope_phases([0.5, bad], device="cpu")


def test_phases_of_nothing():
    assert blkattn.rope_phases([], device="cpu").shape == (0,)


def test_angles_plain_linear_base():
    rot, base, f = 64, 10000.0, 4.0
    plain, m = blkattn.rope_angles(rot, base)
    assert m == 1.0 and len(plain) == 32
    for i, w in enumerate(plain):
        assert w == pytest.approx(base ** (-2 * i / rot), rel=1e-14)
    linear, _ = blkattn.rope_angles(rot, base, "linear", factor=f)
    assert all(a == pytest.approx(b / f, rel=1e-14) for a, b in zip(linear, plain))
    based, _ = blkattn.rope_angles(rot, base, "base", factor=f)
    assert based[0] == plain[0]
    assert based[-1] == pytest.approx(plain[-1] / f, rel=1e-12)  # the slowest pair turns `factor` times slower


def test_angles_ramp():
    rot, base, f, L = 128, 10000.0, 8.0, 8192.0
    plain, _ = blkattn.rope_angles(rot, base)
    ramp, m = blkattn.rope_angles(rot, base, "ramp", factor=f, trained=L, low=1.0, high=32.0)
    assert m == pytest.approx(0.1 * math.log(f) + 1.0, rel=1e-6)
    kept = divided = between = 0
    for a, w in zip(ramp, plain):
        turns = L * w / (2 * math.pi)
        if turns >= 32:
            assert a == pytest.approx(w, rel=1e-14)
            kept += 1
        elif turns <= 1:
            assert a == pytest.approx(w / f, rel=1e-14)
            divided += 1
        else:
            k = (turns - 1) / 31
            assert a == pytest.approx(k * w + (1 - k) * w / f, rel=1e-12)
            between += 1
    assert kept and divided and between
    assert blkattn.rope_angles(rot, base, "ramp", factor=1.0, trained=L)[0] == pytest.approx(plain, rel=1e-14)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=1026), dict(rot=-2), dict(base=1.0),
                                dict(base=math.nan), dict(base=math.inf), dict(scaling="linear", factor=0.5),
                                dict(scaling="linear", factor=math.nan), dict(scaling="base", factor=2.0, rot=2),
                                dict(scaling="ramp", factor=2.0, trained=0.0),
                                dict(scaling="ramp", factor=2.0, trained=64.0, low=4.0, high=4.0),
                                dict(scaling="ramp", factor=math.inf, trained=64.0), dict(scaling="no such")])
def test_angles_refuse(kw):
    args = dict(rot=64, base=10000.0)
    args.update(kw)
    with pytest.raises(ValueError):
        blkattn.rope_angles(**args)


def test_angles_null(lib):
    spec = blkattn.RopeSpec(64, 0, 10000.0, 1.0, 0.0, 0.0, 1.0)
    assert lib.blkattn_rope_angles(None, None, None) == -1
    assert lib.blkattn_rope_angles(ctypes.byref(spec), None, None) == -1
    w = (ctypes.c_double * 32)()
    assert lib.blkattn_rope_angles(ctypes.byref(spec), w, None) == 0  # mscale may be NULL
    spec.scaling = 9
    assert lib.blkattn_rope_angles(ctypes.byref(spec), w, None) == -1


# --------------------------------------------------------------- refusals
I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


def rope_args():
    return dict(x=FakeTensor((2, 4, 3, 128), BF16), pos=FakeTensor((2, 3), I32), ph=FakeTensor((64,), I64), layout=0,
                mscale=1.0, y=FakeTensor((2, 4, 3, 128), BF16, addr=0x20000))


def call_rope(lib, a, name="blkattn_rope"):
    return getattr(lib, name)(ref(a["x"]), ref(a["pos"]), ref(a["ph"]), a["layout"], a["mscale"], ref(a["y"]), None)


@pytest.mark.parametrize("name", ["blkattn_rope", "blkattn_rope_bwd"])
@pytest.mark.parametrize("change,want", [
    (dict(x=None), -1), (dict(pos=None), -1), (dict(ph=None), -1), (dict(y=None), -1),
    (dict(x=FakeTensor((2, 4, 3, 128), I32)), -1),
    (dict(y=FakeTensor((2, 4, 3, 128), I64, addr=0x20000)), -1),
    (dict(x=FakeTensor((4, 3, 128), BF16)), -1),
    (dict(y=FakeTensor((2, 4, 3, 64), BF16, addr=0x20000)), -1),
    (dict(pos=FakeTensor((2, 3), I64)), -1), (dict(pos=FakeTensor((2, 4), I32)), -1),
    (dict(ph=FakeTensor((64,), F32)), -1), (dict(ph=FakeTensor((0,), I64)), -1), (dict(ph=FakeTensor((65,), I64)), -1),
    (dict(layout=2), -1), (dict(layout=-1), -1), (dict(mscale=math.nan), -1), (dict(mscale=math.inf), -1),
    (dict(y=FakeTensor((2, 4, 3, 128), BF16, strides=(1536, 0, 128, 1), addr=0x20000)), -1),  # written through a broadcast
    (dict(y=FakeTensor((2, 4, 3, 128), BF16, strides=(1536, 128, 512, 1), addr=0x10000)), -1),  # x's memory, another view
    (dict(y=FakeTensor((2, 4, 3, 128), F32, addr=0x10000)), -1),                                # x's memory, another type
    (dict(x=FakeTensor((2, 4, 3, 128), BF16, strides=(1536, 384, -128, 1))), -1),
    (dict(x=FakeTensor((2, 4, 3, 128), BF16, device=1)), -1), (dict(pos=FakeTensor((2, 3), I32, device=-1)), -1),
    (dict(x=FakeTensor((2, 4, 3, 128), BF16, addr=None)), -1), (dict(ph=FakeTensor((64,), I64, addr=None)), -1),
    (dict(x=FakeTensor((2, 4, 3, 1026), BF16), y=FakeTensor((2, 4, 3, 1026), BF16, addr=0x90000)), -2),
    (dict(x=FakeTensor((2, 70000, 3, 128), BF16), y=FakeTensor((2, 70000, 3, 128), BF16, addr=0x90000)), -2),
])
def test_rope_refuses(lib, name, change, want):
    a = rope_args()
    a.update(change)
    assert call_rope(lib, a, name) == want


def test_rope_of_no_rows_is_a_no_op(lib):
    for shape in ((0, 4, 3, 128), (2, 0, 3, 128), (2, 4, 0, 128)):
        a = rope_args()
        a.update(x=FakeTensor(shape, BF16, addr=None), y=FakeTensor(shape, BF16, addr=None),
                 pos=FakeTensor((shape[0], shape[2]), I32, addr=None))
        assert call_rope(lib, a) == 0


def append_args(T=3, page=16, N=7, entries=5, dt=BF16):
    return dict(k=FakeTensor((2, 4, T, 128), dt), v=FakeTensor((2, 4, T, 128), dt), pos=FakeTensor((2, T), I32),
                table=FakeTensor((2, entries), I32), kp=FakeTensor((N, 4, page, 128), dt, addr=0x100000),
                vp=FakeTensor((N, 4, page, 128), dt, addr=0x200000), ph=FakeTensor((64,), I64), layout=0, mscale=1.0,
                q=FakeTensor((2, 8, T, 128), dt), qo=FakeTensor((2, 8, T, 128), dt, addr=0x300000))


def call_append(lib, a):
    return lib.blkattn_paged_append(ref(a["k"]), ref(a["v"]), ref(a["pos"]), ref(a["table"]), ref(a["kp"]),
                                    ref(a["vp"]), ref(a["ph"]), a["layout"], a["mscale"], ref(a["q"]), ref(a["qo"]),
                                    None)


@pytest.mark.parametrize("change,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(pos=None), -1), (dict(table=None), -1), (dict(kp=None), -1),
    (dict(vp=None), -1), (dict(q=None), -1), (dict(qo=None), -1),
    (dict(v=FakeTensor((2, 4, 3, 128), F32)), -1), (dict(v=FakeTensor((2, 4, 3, 64), BF16)), -1),
    (dict(kp=FakeTensor((7, 4, 16, 128), F32, addr=0x100000)), -1),
    (dict(kp=FakeTensor((7, 5, 16, 128), BF16, addr=0x100000)), -1),
    (dict(kp=FakeTensor((8, 4, 16, 128), BF16, addr=0x100000)), -1),   # pools of two sizes
    (dict(kp=FakeTensor((7, 4, 16, 128), BF16, strides=(0, 2048, 128, 1), addr=0x100000)), -1),
    (dict(kp=FakeTensor((7, 4, 16, 128), BF16, addr=0x200000)), -1),   # both pools at one address
    (dict(table=FakeTensor((3, 5), I32)), -1), (dict(table=FakeTensor((2, 0), I32)), -1),
    (dict(table=FakeTensor((2, 5), I64)), -1), (dict(pos=FakeTensor((2, 3), I64)), -1),
    (dict(ph=FakeTensor((65,), I64)), -1), (dict(layout=3), -1), (dict(mscale=math.nan), -1),
    (dict(qo=FakeTensor((2, 8, 3, 128), F32, addr=0x300000)), -1),
    (dict(qo=FakeTensor((2, 8, 3, 128), BF16, strides=(1024, 0, 128, 1), addr=0x300000)), -1),
    (dict(q=FakeTensor((2, 8, 4, 128), BF16)), -1), (dict(table=FakeTensor((2, 5), I32, device=1)), -1),
    (dict(vp=FakeTensor((7, 4, 16, 128), BF16, addr=None)), -1), (dict(qo=FakeTensor((2, 8, 3, 128), BF16, addr=None)), -1),
    (dict(table=FakeTensor((2, 1 << 27), I32)), -2),   # 2^31 cache rows a sequence
])
def test_append_refuses(lib, change, want):
    a = append_args()
    a.update(change)
    assert call_append(lib, a) == want


@pytest.mark.parametrize("page,want", [(0, -1), (4, -2), (24, -2), (100, -2), (1 << 17, -2)])
def test_append_refuses_page_sizes(lib, page, want):
    assert call_append(lib, append_args(page=page)) == want


def test_append_of_no_rows_is_a_no_op(lib):
    a = append_args(T=0)
    for n in ("k", "v", "q", "qo", "pos"):
        a[n].addr = None
    assert call_append(lib, a) == 0


def test_binding_refuses_by_name():
    x = torch.zeros(1, 1, 1, 8)
    with pytest.raises(ValueError):
        blkattn.rope(x, torch.zeros(1, 1, dtype=I32), torch.zeros(4, dtype=I64), layout="neither")
    with pytest.raises(ValueError):  # host memory
        blkattn.rope(x, torch.zeros(1, 1, dtype=I32), torch.zeros(4, dtype=I64))
    with pytest.raises(ValueError):
        blkattn.rope(x.double(), torch.zeros(1, 1, dtype=I32), torch.zeros(4, dtype=I64))


def test_binding_refuses_what_is_no_tensor():
    x, pos, ph = torch.zeros(1, 1, 1, 8), torch.zeros(1, 1, dtype=I32), torch.zeros(4, dtype=I64)
    with pytest.raises(TypeError):
        blkattn.rope(3.0, pos, ph)
    with pytest.raises(TypeError):
        blkattn.rope(x, "pos", ph)
    with pytest.raises(TypeError):
        blkattn.rope(x, pos, ph, out_dtype="float")
    with pytest.raises(ValueError):
        blkattn.rope(torch.zeros(1, 1, 1, 1, 8), pos, ph)  # five dimensions
    with pytest.raises(ValueError):
        blkattn.rope(x.to_sparse(), pos, ph)
    with pytest.raises(ValueError):
        blkattn.rope(x, pos, None)  # a missing argument is the library's refusal
