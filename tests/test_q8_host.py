"""Host-side checks of the head norms and of the 8-bit cache: refusals come before any CUDA call.  No GPU."""
import ctypes
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn
from exact_blocked_attention_gb300 import build as libbuild

from test_abi_host import FakeTensor

I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Fake(FakeTensor):
    """FakeTensor of any dtype of the binding."""

    def desc(self):
        kept, self.dtype = self.dtype, I32
        d = super().desc()
        self.dtype = kept
        d.dtype = blkattn._DTYPES[kept]
        return d


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return blkattn.load()


def ref(t):
    return None if t is None else ctypes.byref(t.desc())


def change(a, what):
    a.update(what)
    return a


# ---------------------------------------------------------------- head norms
def norm_args(B=2, Hq=8, Hk=2, T=3, d=128, rot=128, dt=BF16):
    return dict(q=Fake((B, Hq, T, d), dt), wq=Fake((d,), BF16), k=Fake((B, Hk, T, d), dt, addr=0x200000),
                wk=Fake((d,), BF16), pos=Fake((B, T), I32), ph=Fake((rot // 2,), I64) if rot else None, layout=0,
                mscale=1.0, eps=1e-6, qo=Fake((B, Hq, T, d), dt, addr=0x300000), ko=Fake((B, Hk, T, d), dt, addr=0x400000),
                gq=Fake((B, Hq, T, d), F32), gk=Fake((B, Hk, T, d), F32), dwq=Fake((d,), F32, addr=0x500000),
                dwk=Fake((d,), F32, addr=0x600000))


def norm(lib, a):
    return lib.blkattn_qk_norm_rope(ref(a["q"]), ref(a["wq"]), ref(a["k"]), ref(a["wk"]), ref(a["pos"]), ref(a["ph"]),
                                    a["layout"], a["mscale"], a["eps"], ref(a["qo"]), ref(a["ko"]), None)


def norm_bwd(lib, a):
    return lib.blkattn_qk_norm_rope_bwd(ref(a["gq"]), ref(a["gk"]), ref(a["q"]), ref(a["wq"]), ref(a["k"]), ref(a["wk"]),
                                        ref(a["pos"]), ref(a["ph"]), a["layout"], a["mscale"], a["eps"], ref(a["qo"]),
                                        ref(a["ko"]), ref(a["dwq"]), ref(a["dwk"]), None)


NORM = [
    dict(q=None), dict(wq=None), dict(pos=None), dict(qo=None), dict(k=None), dict(wk=None), dict(ko=None),
    dict(wq=Fake((64,), BF16)), dict(wq=Fake((128,), I32)), dict(wk=Fake((128,), F32)),
    dict(k=Fake((2, 2, 3, 64), BF16)), dict(k=Fake((2, 2, 4, 128), BF16)), dict(k=Fake((2, 2, 3, 128), F32)),
    dict(qo=Fake((2, 8, 4, 128), BF16)), dict(qo=Fake((2, 8, 3, 128), F32)), dict(qo=Fake((2, 8, 3, 128), I32)),
    dict(qo=Fake((2, 8, 3, 128), BF16, strides=(4096, 0, 128, 1))),
    dict(pos=Fake((2, 4), I32)), dict(pos=Fake((2, 3), I64)), dict(ph=Fake((65,), I64)), dict(ph=Fake((64,), I32)),
    dict(ph=Fake((0,), I64)), dict(layout=2), dict(mscale=math.inf), dict(eps=math.nan), dict(eps=-1e-6),
    dict(pos=Fake((2, 3), I32, device=1)), dict(wk=Fake((128,), BF16, device=1)), dict(q=Fake((2, 8, 3, 128), BF16, device=-1)),
    dict(qo=Fake((2, 8, 3, 128), BF16, addr=None)), dict(wq=Fake((128,), BF16, addr=None)), dict(ph=Fake((64,), I64, addr=None)),
    dict(qo=Fake((2, 8, 3, 128), BF16, addr=0x400000)),  # both outputs in one place
]


@pytest.mark.parametrize("what", NORM)
def test_norm_refuses(lib, what):
    assert norm(lib, change(norm_args(), what)) == -1


@pytest.mark.parametrize("what", NORM + [
    dict(gq=None), dict(gk=None), dict(dwq=None), dict(dwk=None), dict(dwq=Fake((128,), BF16)), dict(dwq=Fake((64,), F32)),
    dict(dwq=Fake((128,), F32, strides=(0,))), dict(dwk=Fake((128,), F32, addr=0x500000)), dict(gk=Fake((2, 2, 3, 128), BF16)),
    dict(gq=Fake((2, 7, 3, 128), F32)), dict(dwq=Fake((128,), F32, addr=None))])
def test_norm_bwd_refuses(lib, what):
    assert norm_bwd(lib, change(norm_args(), what)) == -1


def test_norm_sizes(lib):
    for kw in (dict(d=1025, rot=0), dict(Hq=1 << 15), dict(B=1 << 16, T=1 << 16), dict(B=1 << 10, T=1 << 10, Hq=1 << 13)):
        assert norm(lib, norm_args(**kw)) == -2 and norm_bwd(lib, norm_args(**kw)) == -2
    for kw in (dict(B=0), dict(T=0), dict(Hq=0, Hk=0)):
        a = norm_args(**kw)
        for n in ("q", "k", "qo", "ko", "pos"):
            a[n].addr = None
        assert norm(lib, a) == 0
    a = norm_args()
    a["k"] = a["wk"] = a["ko"] = None
    a["wq"].addr = None
    assert norm(lib, a) == -1  # (k may be left out, a weight not)


# ---------------------------------------------------------------- the 8-bit cache
def cache(B=2, Hkv=2, d=128, P=16, S=8, N=9, entries=4):
    return dict(table=Fake((B, entries), I32), kp=Fake((N, Hkv, P, d), F8, addr=0x100000),
                vp=Fake((N, Hkv, P, d), F8, addr=0x200000), ks=Fake((N, Hkv, max(1, P // S)), E8, addr=0x300000),
                vs=Fake((N, Hkv, max(1, P // S)), E8, addr=0x400000))


def append_args(B=2, Hq=8, Hkv=2, T=3, d=128, dt=BF16, **kw):
    return dict(k=Fake((B, Hkv, T, d), dt), v=Fake((B, Hkv, T, d), dt), pos=Fake((B, T), I32), q=Fake((B, Hq, T, d), dt),
                qo=Fake((B, Hq, T, d), dt, addr=0x600000), wk=Fake((d,), F32), wq=Fake((d,), F32), eps=1e-6,
                ph=Fake((d // 2,), I64), layout=0, mscale=1.0, **cache(B, Hkv, d, **kw))


def append(lib, a):
    return lib.blkattn_paged_append_q8(ref(a["k"]), ref(a["v"]), ref(a["pos"]), ref(a["table"]), ref(a["kp"]), ref(a["vp"]),
                                       ref(a["ks"]), ref(a["vs"]), ref(a["wk"]), a["eps"], ref(a["ph"]), a["layout"],
                                       a["mscale"], ref(a["q"]), ref(a["wq"]), ref(a["qo"]), None)


def read_args(B=2, Hkv=2, T=3, d=128, **kw):
    return dict(pos=Fake((B, T), I32), ko=Fake((B, Hkv, T, d), BF16, addr=0x600000),
                vo=Fake((B, Hkv, T, d), BF16, addr=0x700000), **cache(B, Hkv, d, **kw))


def read(lib, a):
    return lib.blkattn_paged_read_q8(ref(a["pos"]), ref(a["table"]), ref(a["kp"]), ref(a["vp"]), ref(a["ks"]), ref(a["vs"]),
                                     ref(a["ko"]), ref(a["vo"]), None)


def fwd_args(B=2, Hq=8, Hkv=2, Tq=3, d=128, **kw):
    return dict(q=Fake((B, Hq, Tq, d), BF16), sl=Fake((B,), I32), qp=Fake((B, Tq), I32), tree=None, window=0, scale=0.1,
                out=Fake((B, Hq, Tq, d), F32, addr=0x600000), lse=Fake((B, Hq, Tq), F32, addr=0x700000),
                **cache(B, Hkv, d, **kw))


def fwd(lib, a):
    return lib.blkattn_fwd_paged_q8(ref(a["q"]), ref(a["kp"]), ref(a["vp"]), ref(a["ks"]), ref(a["vs"]), ref(a["table"]),
                                    ref(a["sl"]), ref(a["qp"]), ref(a["tree"]), a["window"], a["scale"], ref(a["out"]),
                                    ref(a["lse"]), None)


CACHE = [
    (dict(kp=None), -1), (dict(vp=None), -1), (dict(ks=None), -1), (dict(vs=None), -1), (dict(table=None), -1),
    (dict(kp=Fake((9, 2, 16, 128), BF16, addr=0x100000)), -1), (dict(vp=Fake((9, 2, 16, 128), E8, addr=0x200000)), -1),
    (dict(kp=Fake((8, 2, 16, 128), F8, addr=0x100000)), -1), (dict(ks=Fake((9, 2, 2), F32)), -1),
    (dict(ks=Fake((9, 2, 2), F8)), -1), (dict(ks=Fake((9, 2, 3), E8)), -1), (dict(ks=Fake((9, 2, 0), E8)), -1),
    (dict(ks=Fake((9, 2, 32), E8), vs=Fake((9, 2, 32), E8)), -1), (dict(vs=Fake((9, 2, 4), E8, addr=0x400000)), -1),
    (dict(ks=Fake((8, 2, 2), E8)), -1), (dict(ks=Fake((9, 1, 2), E8)), -1), (dict(ks=Fake((9, 2), E8)), -1),
    (dict(ks=Fake((9, 2, 2), E8, strides=(4, 0, 1))), -1),
    (dict(kp=Fake((9, 2, 16, 128), F8, strides=(4096, 2048, 128, 2), addr=0x100000)), -1),
    (dict(kp=Fake((9, 2, 16, 128), F8, strides=(4096, 2048, 136, 1), addr=0x100000)), -1),
    (dict(vp=Fake((9, 2, 16, 128), F8, strides=(4096, 0, 128, 1), addr=0x200000)), -1),
    (dict(vp=Fake((9, 2, 16, 128), F8, addr=0x200008)), -1),
    (dict(kp=Fake((9, 2, 16, 128), F8, addr=None)), -1), (dict(vs=Fake((9, 2, 2), E8, addr=None)), -1),
    (dict(table=Fake((2, 4), I64)), -1), (dict(table=Fake((2, 4), I32, addr=None)), -1),
    (dict(table=Fake((2, 4), I32, device=1)), -1), (dict(ks=Fake((9, 2, 2), E8, device=1)), -1),
]


@pytest.mark.parametrize("what,want", CACHE + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(pos=None), -1), (dict(v=Fake((2, 2, 3, 128), F32)), -1),
    (dict(v=Fake((2, 2, 4, 128), BF16)), -1), (dict(k=Fake((2, 2, 3, 128), I32)), -1), (dict(pos=Fake((2, 3), I64)), -1),
    (dict(q=None), -1), (dict(qo=None), -1), (dict(q=None, qo=None), -1),  # a q_weight without q
    (dict(qo=Fake((2, 8, 3, 128), F32)), -1), (dict(q=Fake((2, 8, 3, 64), BF16)), -1),
    (dict(qo=Fake((2, 8, 3, 128), BF16, strides=(4096, 0, 128, 1))), -1),
    (dict(wk=Fake((64,), F32)), -1), (dict(wk=Fake((128,), BF16)), -1), (dict(wq=Fake((128,), I32)), -1), (dict(eps=-1.0), -1),
    (dict(eps=math.nan), -1), (dict(wk=Fake((128,), F32, addr=None)), -1), (dict(ph=Fake((65,), I64)), -1), (dict(layout=7), -1),
    (dict(mscale=math.nan), -1), (dict(vp=Fake((9, 2, 16, 128), F8, addr=0x100000)), -1),
    (dict(vs=Fake((9, 2, 2), E8, addr=0x300000)), -1)])
def test_append_refuses(lib, what, want):
    assert append(lib, change(append_args(), what)) == want


@pytest.mark.parametrize("what,want", CACHE + [
    (dict(pos=None), -1), (dict(ko=None), -1), (dict(vo=None), -1), (dict(vo=Fake((2, 2, 3, 128), F32)), -1),
    (dict(ko=Fake((2, 2, 3, 128), F8), vo=Fake((2, 2, 3, 128), F8)), -1), (dict(pos=Fake((2, 4), I32)), -1),
    (dict(vo=Fake((2, 2, 3, 128), BF16, addr=0x600000)), -1),
    (dict(ko=Fake((2, 2, 3, 128), BF16, strides=(0, 384, 128, 1))), -1)])
def test_read_refuses(lib, what, want):
    assert read(lib, change(read_args(), what)) == want


@pytest.mark.parametrize("what,want", CACHE + [
    (dict(q=None), -1), (dict(sl=None), -1), (dict(qp=None), -1), (dict(out=None), -1), (dict(lse=None), -1),
    (dict(q=Fake((2, 8, 3, 128), F32)), -2), (dict(q=Fake((2, 8, 3, 128), F8)), -1), (dict(q=Fake((2, 9, 3, 128), BF16)), -1),
    (dict(out=Fake((2, 8, 3, 128), F8)), -1), (dict(window=-1), -1), (dict(window=1 << 31), -1), (dict(scale=math.nan), -1),
    (dict(tree=Fake((2, 3), I32)), -1), (dict(window=4, tree=Fake((2, 3), I64)), -1),
    (dict(out=Fake((2, 8, 3, 128), F32, strides=(1024, 0, 128, 1))), -1), (dict(sl=Fake((2,), I64)), -1)])
def test_fwd_refuses(lib, what, want):
    assert fwd(lib, change(fwd_args(), what)) == want


@pytest.mark.parametrize("kw,want", [(dict(P=4, S=4), -2), (dict(P=48, S=48), -2), (dict(P=256, S=256), -2), (dict(d=96), -2),
                                     (dict(d=256), -2), (dict(N=0), -1), (dict(entries=0), -1)])
def test_refuses_sizes(lib, kw, want):
    assert append(lib, append_args(**kw)) == want
    assert read(lib, read_args(**kw)) == want
    assert fwd(lib, fwd_args(**kw)) == want


@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0)])
def test_no_rows_is_a_no_op(lib, kw):
    a = append_args(**kw)
    for n in ("k", "v", "pos", "q", "qo"):
        a[n].addr = None
    b = read_args(**kw)
    for n in ("pos", "ko", "vo"):
        b[n].addr = None
    kw = {"Tq" if n == "T" else n: v for n, v in kw.items()}
    c = fwd_args(**kw)
    for n in ("q", "sl", "qp", "out", "lse"):
        c[n].addr = None
    if kw.get("B") == 0:
        for x in (a, b, c):
            x["table"].addr = None
    assert append(lib, a) == 0 and read(lib, b) == 0 and fwd(lib, c) == 0


def test_pools_too_far_apart_for_attention(lib):
    """Rows of a head more than 64 GiB from the first: the attention kernels keep 32 bits of 16 bytes."""
    far = Fake((9, 2, 16, 128), F8, strides=(1 << 33, 2048, 128, 1), addr=0x100000)
    near = Fake((9, 2, 16, 128), F8, strides=((1 << 33) - 1024, 2048, 128, 1), addr=0x100000)
    for n in ("kp", "vp"):
        assert fwd(lib, change(fwd_args(), {n: far})) == -2
    assert fwd(lib, change(fwd_args(), {"kp": near, "sl": Fake((2,), I32, addr=None)})) == -1  # (as far as the next check)
