"""The 8-bit paged cache on the GPU: the append and the read against their
definition in 64 bits.

Without norm and rotation everything is exact: bytes and exponents equal the
definition's.  With them a number is off by what test_gpu_qk_norm.py derives
before it is rounded to e4m3 (half a step, 2^-4 of the value or 2^-10 of the
block's scale), and a block's exponent may be the next one where its largest
number lies within that bound of 448 2^e.
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_qk_norm import EPS, n_of, normed
from test_gpu_rotary import angles, check, dev, pairs, turned

pytestmark = pytest.mark.gpu
BF16, F32, F64, U8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def exponent(amax: float) -> int:
    if amax == 0:
        return -127
    m, ex = math.frexp(amax)
    return max(-127, ex - 9 + (m > 0.875))


def to_e4m3(x):
    """Values (64 bits, within range) as the e4m3 byte nearest to each, ties to even; NaN for what is not finite."""
    x = torch.where(torch.isfinite(x), x, math.nan)
    k = torch.frexp(x).exponent.clamp(min=-5).double() - 4
    return (torch.round(x * torch.exp2(-k)) * torch.exp2(k)).float().to(F8)


def pools(N, H, P, d, S, seed=0, rows_major=False):
    """Two random pools: any bytes but NaN, exponents of a few sizes."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        b = torch.randint(0, 256, (N, H, P, d), generator=g).to(U8)
        b[(b & 0x7f) == 0x7f] = 0x30
        s = torch.randint(115, 125, (N, H, P // S), generator=g).to(U8)
        b = b.to(dev())
        if rows_major:
            b = b.transpose(1, 2).contiguous().transpose(1, 2)
        out += [b.view(F8), s.to(dev()).view(E8)]
    return out[0], out[2], out[1], out[3]  # k, v, k_scales, v_scales


def problem(B, Hq, Hkv, T, d, P, S, starts, news=None, dtype=BF16, seed=0, rows_major=False, token_major=True, lead=0):
    """New rows at positions starts[b] ..; lead: rows of padding before them."""
    g = torch.Generator().manual_seed(seed)
    news = news or [T - lead] * B
    entries = max(-(-(s + n) // P) for s, n in zip(starts, news)) + 1
    N = B * entries + 2
    table = torch.randperm(N, generator=g)[:B * entries].to(I32).reshape(B, entries)
    pos = torch.full((B, T), -1, dtype=I32)
    for b in range(B):
        pos[b, lead:lead + news[b]] = torch.arange(starts[b], starts[b] + news[b], dtype=I32)

    def rows(H):
        x = torch.randn(B, T, H, d, generator=g) * torch.exp(2 * torch.randn(B, T, H, 1, generator=g))
        x = x.to(dtype).to(dev())
        return x.transpose(1, 2) if token_major else x.transpose(1, 2).contiguous()

    kp, vp, ks, vs = pools(N, Hkv, P, d, S, seed + 1, rows_major)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(BF16).to(dev()) for _ in range(2)]
    return dict(k=rows(Hkv), v=rows(Hkv), q=rows(Hq), pos=pos.to(dev()), table=table.to(dev()), kp=kp, vp=vp, ks=ks,
                vs=vs, wq=w[0], wk=w[1], P=P, S=S)


def call(a, ph=None, norm=False, **kw):
    return blkattn.paged_append_q8(a["k"], a["v"], a["pos"], a["table"], a["kp"], a["vp"], a["ks"], a["vs"], phases=ph,
                                   k_weight=a["wk"] if norm else None, q_weight=a["wq"] if norm else None, eps=EPS,
                                   q=a["q"], **kw)


def snapshot(a):
    return {n: a[n].view(U8).cpu().clone() for n in ("kp", "vp", "ks", "vs")}


def expect(a, before, rows, slack, pool, scales):
    """What rows [B, H, T, d] (64 bits, each off by at most slack before it is rounded) leave in a pool: checks the
    pool on the GPU against it.  Returns the number of blocks whose exponent the slack decided."""
    P, S = a["P"], a["S"]
    got, gots = a[pool].view(U8).cpu(), a[scales].view(U8).cpu()
    old, olds = before[pool], before[scales]
    touched = torch.zeros(got.shape[:3], dtype=torch.bool)
    moved = torch.zeros(gots.shape, dtype=torch.bool)
    pos, table = a["pos"].cpu(), a["table"].cpu()
    N = got.shape[0]
    either = 0
    for b in range(pos.shape[0]):
        new = {}
        for t, p in enumerate(pos[b].tolist()):
            if p >= 0 and p // P < table.shape[1] and 0 <= int(table[b, p // P]) < N:
                new.setdefault(p // S, {})[p % S] = t  # (the last of several)
        for blk, members in new.items():
            page, row0 = int(table[b, blk * S // P]), blk * S % P
            i = row0 // S
            rs, ts = list(members), [members[r] for r in members]
            x, dx = rows[b][:, ts], slack[b][:, ts]
            for h in range(got.shape[1]):
                fin = torch.isfinite(x[h])
                size = torch.where(fin, x[h].abs(), 0.0)
                lo, hi = (float(torch.where(fin, (size + f * dx[h]).clamp(min=0), 0.0).max()) for f in (-1, 1))
                e_old = int(olds[page, h, i]) - 127
                cand = {e if 0 in members else max(e, e_old) for e in (exponent(lo), exponent(hi))}
                e = int(gots[page, h, i]) - 127
                assert e in cand, (b, blk, h, e, cand)
                either += len(cand) > 1
                f = 2.0 ** -e
                want = x[h] * f
                have = got[page, h][[row0 + r for r in rs]].view(F8).double()
                if bool((dx == 0).all()):
                    assert torch.equal(to_e4m3(want).double().nan_to_num(nan=1e9), have.nan_to_num(nan=1e9))
                else:
                    bound = dx[h] * f * (1 + 2.0 ** -4) + torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10, dtype=F64))
                    assert bool(((have - want).abs() <= bound).all())
                rest = [r for r in range(S) if r not in members]
                o = old[page, h][[row0 + r for r in rest]]
                if 0 not in members and e > e_old:
                    o = to_e4m3(o.view(F8).double() * 2.0 ** (e_old - e)).view(U8)
                assert torch.equal(got[page, h][[row0 + r for r in rest]].view(F8).float(), o.view(F8).float())
            touched[page, :, row0:row0 + S] = True
            moved[page, :, i] = True
    assert torch.equal(got[~touched], old[~touched]) and torch.equal(gots[~moved], olds[~moved])
    return either


APPEND = [
    dict(B=3, Hq=4, Hkv=2, T=1, d=128, P=16, S=16, starts=[0, 5, 31]),
    dict(B=2, Hq=33, Hkv=5, T=1, d=64, P=8, S=8, starts=[7, 16]),
    dict(B=2, Hq=2, Hkv=1, T=37, d=128, P=16, S=4, starts=[3, 0]),
    dict(B=2, Hq=3, Hkv=3, T=50, d=64, P=32, S=1, starts=[0, 9], dtype=F32),
    dict(B=2, Hq=8, Hkv=2, T=150, d=128, P=64, S=32, starts=[1, 60], news=[150, 33]),
    dict(B=1, Hq=2, Hkv=2, T=300, d=128, P=128, S=128, starts=[100], rows_major=True),
    dict(B=1, Hq=2, Hkv=2, T=200, d=64, P=256, S=64, starts=[40], dtype=F32, token_major=False),
    dict(B=2, Hq=1, Hkv=1, T=90, d=128, P=16, S=2, starts=[0, 1], news=[3, 20], lead=70),
    dict(B=1, Hq=4, Hkv=1, T=17, d=64, P=16, S=16, starts=[15], rows_major=True),
]


def ident(c):
    return "-".join(str(v).replace("torch.", "") for v in c.values())


@pytest.mark.parametrize("case", APPEND, ids=ident)
def test_append_exact(case):
    a = problem(**case)
    before = snapshot(a)
    q_out = call(a)
    zero = torch.zeros(a["k"].shape, dtype=F64)
    for rows, pool, scales in (("k", "kp", "ks"), ("v", "vp", "vs")):
        expect(a, before, a[rows].double().cpu(), zero, pool, scales)
    keep = (a["pos"] >= 0)[:, None, :, None]
    assert torch.equal(q_out, torch.where(keep, a["q"], 0.0))


@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 32), ("half", 22), ("interleaved", 10)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", APPEND, ids=ident)
def test_append_normed_and_turned(case, norm, layout, rot):
    a = problem(**case)
    ang = angles(rot)
    before = snapshot(a)
    q_out = call(a, blkattn.rope_phases(ang), norm, layout=layout, mscale=1.1)
    for rows, w, out in (("k", "wk", None), ("q", "wq", q_out)):
        u = normed(a[rows], a[w]) if norm else a[rows].double().cpu()
        y, slack = turned(u, a["pos"], ang, layout, 1.1)
        if norm:
            size = u.abs()
            i, j = pairs(rot, layout)
            size[..., i] = size[..., j] = 1.1 * (u[..., i].abs() + u[..., j].abs())
            slack = slack + n_of(u.shape[-1]) * size
        if out is None:
            expect(a, before, y, slack, "kp", "ks")
        else:
            keep = (a["pos"].cpu() >= 0)[:, None, :, None]
            check(out, torch.where(keep, y, 0.0), torch.where(keep, slack, 0.0))
    expect(a, before, a["v"].double().cpu(), torch.zeros(a["v"].shape, dtype=F64), "vp", "vs")


def test_append_token_by_token():
    """A block filled one row at a time: what the cache stands for stays within the roundings that its rising scale
    costs (each rise may round a row's smallest numbers again, by half of 2^(e - 9) each)."""
    a = problem(1, 1, 2, 1, 128, 32, 16, [0], seed=4)
    g = torch.Generator().manual_seed(8)
    want = torch.randn(1, 2, 32, 128, generator=g) * torch.exp2(torch.arange(32) / 4.0)[:, None]
    want = want.to(BF16)
    for t in range(32):
        a["k"] = want[:, :, t:t + 1].to(dev())
        a["v"] = a["k"].clone()
        a["pos"] = torch.tensor([[t]], dtype=I32, device=dev())
        call(a)
    pos = torch.arange(32, dtype=I32, device=dev())[None]
    k, v = blkattn.paged_read_q8(pos, a["table"], a["kp"], a["vp"], a["ks"], a["vs"], out_dtype=F32)
    assert torch.equal(k, v)
    page = int(a["table"][0, 0])
    e = (a["ks"].view(U8)[page].double().cpu() - 127).repeat_interleave(16, 1)[None, :, :, None]  # [1, 2, 32, 1]
    # one rounding of 2^-4, and at most 16 more of half the grid's step below 2^-6 2^e (exact above it)
    bound = 2.0 ** -4 * want.double().abs() + 17 * torch.exp2(e - 10)
    assert bool(((k.double().cpu() - want.double()).abs() <= bound).all())


def test_append_odd_rows():
    """Infinities and NaN are stored as NaN and leave the scale to the others; zeros, the smallest and the largest
    numbers; the same row twice (the last stays); rows without a page, past the table, and padding."""
    a = problem(1, 1, 1, 40, 64, 16, 8, [0], seed=2)
    a["k"][0, 0, 3, 7] = math.nan
    a["k"][0, 0, 4, 9] = math.inf
    a["v"][0, 0, 5, 1] = -math.inf
    a["k"][0, 0, 8:16] = 0
    a["v"][0, 0, 8:16] = 2.0 ** -130
    a["k"][0, 0, 16:24] = 3e38
    a["v"][0, 0, 16:20] = math.nan
    a["v"][0, 0, 20:24] = math.inf
    a["pos"][0, 26] = a["pos"][0, 25]
    a["table"][0, 1] = -1
    a["table"][0, 2] = 10 ** 9
    a["pos"][0, 39] = 2 ** 31 - 1
    before = snapshot(a)
    call(a)
    zero = torch.zeros(a["k"].shape, dtype=F64)
    expect(a, before, a["k"].double().cpu(), zero, "kp", "ks")
    expect(a, before, a["v"].double().cpu(), zero, "vp", "vs")
    a["table"][0, 1] = int(a["table"][0, 0]) ^ 1
    before = snapshot(a)
    call(a)
    expect(a, before, a["k"].double().cpu(), zero, "kp", "ks")
    expect(a, before, a["v"].double().cpu(), zero, "vp", "vs")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("B,H,T,d,P,S,rows_major", [(3, 2, 70, 128, 16, 4, False), (1, 5, 333, 64, 32, 32, True),
                                                   (2, 1, 1, 128, 8, 1, False), (1, 1, 1000, 64, 256, 128, False)])
def test_read(B, H, T, d, P, S, rows_major, out):
    kp, vp, ks, vs = pools(40, H, P, d, S, 3, rows_major)
    g = torch.Generator().manual_seed(1)
    table = torch.randint(-1, 41, (B, 6), generator=g).to(I32)
    pos = torch.randint(-3, 7 * P, (B, T), generator=g).to(I32)
    ks.view(U8)[5, 0, 0] = 255  # a scale of NaN
    ks.view(U8)[6, 0, 0] = 0    # the smallest
    kp.view(U8)[7, 0, 0, 3] = 0x7f
    got = blkattn.paged_read_q8(pos.to(dev()), table.to(dev()), kp, vp, ks, vs, out_dtype=out)
    wide = torch.full((B, T, H, d + 8), 7.0, dtype=out, device=dev())
    view = wide.transpose(1, 2)[..., :d]
    blkattn.paged_read_q8(pos.to(dev()), table.to(dev()), kp, vp, ks, vs, k_out=view, v_out=torch.empty_like(view))
    assert bool((wide[..., d:] == 7).all())
    for x, pool, scales in ((got[0], kp, ks), (got[1], vp, vs), (view, kp, ks)):
        want = torch.zeros(B, H, T, d, dtype=F64)
        p8, s8 = pool.cpu().float().double(), scales.view(U8).cpu()
        for b in range(B):
            for t in range(T):
                c = int(pos[b, t])
                page = int(table[b, c // P]) if 0 <= c < 6 * P else -1
                if 0 <= page < 40:
                    byte = s8[page, :, c % P // S].double()
                    s = torch.where(byte == 255, math.nan, torch.exp2(byte - 127))
                    want[b, :, t] = p8[page, :, c % P] * s[:, None]
        assert torch.equal(x.double().cpu().nan_to_num(nan=1e9), want.to(out).double().nan_to_num(nan=1e9))


def test_captured_and_replayed():
    a = problem(2, 4, 2, 20, 128, 16, 8, [0, 8])
    before = snapshot(a)
    want_q = call(a, norm=True).clone()
    want = snapshot(a)
    pos = a["pos"]
    read = blkattn.paged_read_q8(pos, a["table"], a["kp"], a["vp"], a["ks"], a["vs"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    q_out = torch.zeros_like(want_q)
    with torch.cuda.graph(graph):
        call(a, norm=True, q_out=q_out)
        got = blkattn.paged_read_q8(pos, a["table"], a["kp"], a["vp"], a["ks"], a["vs"])
    for n, t in before.items():
        a[n].view(U8).copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, want_q) and all(torch.equal(x, y) for x, y in zip(got, read))
    assert all(torch.equal(x, y) for x, y in zip(snapshot(a).values(), want.values()))


@pytest.mark.parametrize("rot,norm", [(128, True), (128, False), (0, True), (0, False), (24, True)])
def test_many_query_rows(rot, norm):
    """Query rows enough for a kernel of their own, with padding in front, behind and between."""
    a = problem(2, 24, 1, 400, 128, 16, 16, [5, 40], news=[300, 250], lead=30)
    a["pos"][0, 100:117] = -1
    ang = angles(rot) if rot else []
    q_out = torch.full_like(a["q"], 7.0)
    before = snapshot(a)
    call(a, blkattn.rope_phases(ang) if ang else None, norm, q_out=q_out)
    u = normed(a["q"], a["wq"]) if norm else a["q"].double().cpu()
    y, slack = turned(u, a["pos"], ang, "half")
    if norm:
        size = u.abs()
        if ang:
            i, j = pairs(rot, "half")
            size[..., i] = size[..., j] = u[..., i].abs() + u[..., j].abs()
        slack = slack + n_of(128) * size
    keep = (a["pos"].cpu() >= 0)[:, None, :, None]
    check(q_out, torch.where(keep, y, 7.0), torch.where(keep, slack, 0.0))
    if not ang and not norm:
        expect(a, before, a["k"].double().cpu(), torch.zeros(a["k"].shape, dtype=F64), "kp", "ks")
