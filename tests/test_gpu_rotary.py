"""Rotary positions and the paged append on the GPU, against 64-bit torch on
the CPU.

Tolerance, derived from the kernel's arithmetic: the angle is a fraction of a
half turn rounded to a float (2^-24 relative, at most pi 2^-24 = 1.9e-7 rad)
plus the table's 2^-63 |t| turns and 2^-32 turns of truncation (2^31 positions:
3e-9 rad); sine and cosine add 2 units in the last place (2.4e-7 at most), the
products and the sum three roundings of 2^-24.  An element is off by at most
(1.9e-7 + 3e-9 + 2.4e-7 + 1.8e-7) (|x_a| + |x_b|) mscale < 6.2e-7 (...), and
a bf16 store adds half a step, 2^-8 of the value (and of that error).
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def dev():
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def angles(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def pairs(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def turned(x, pos, w, layout, mscale=1.0, back=False):
    """(rotated rows, bound before the store) in 64 bits on the CPU; angles reduced with exact integers."""
    x = x.detach().double().cpu()
    y, bound = x.clone(), torch.zeros_like(x)
    if not w:
        return y, bound
    # the exact phase table: whole turns drop out of the wrapping product, however far the position
    table = blkattn.rope_phases(w, device="cpu")
    t = (pos.cpu().long()[:, :, None] * table)  # wraps mod 2^64
    ang = t.double() * (2 * math.pi / 2.0 ** 64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if back:
        s = -s
    a, b = pairs(2 * len(w), layout)
    y[..., a] = mscale * (x[..., a] * c - x[..., b] * s)
    y[..., b] = mscale * (x[..., a] * s + x[..., b] * c)
    bound[..., a] = bound[..., b] = 6.2e-7 * abs(mscale) * (x[..., a].abs() + x[..., b].abs())
    return y, bound


def check(got, want, bound):
    tol = bound
    if got.dtype == BF16:
        tol = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (got.detach().double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def rows(shape, dtype, seed, token_major=False):
    g = torch.Generator().manual_seed(seed)
    B, H, T, d = shape
    x = torch.randn((B, T, H, d) if token_major else shape, generator=g).to(dtype).to(dev())
    return x.transpose(1, 2) if token_major else x


def positions(B, T, seed, far=False):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(-(2 ** 31) if far else 0, 2 ** 31 if far else 4096, (B, T), generator=g).to(torch.int32)
    if far:
        p.view(-1)[0] = 2 ** 31 - 1
        p.view(-1)[-1] = -(2 ** 31)
    return p.to(dev())


SHAPES = [(1, 1, 1, 128, 128), (2, 4, 3, 128, 128), (3, 5, 17, 64, 64), (2, 3, 33, 128, 64), (1, 2, 9, 96, 96),
          (2, 3, 7, 80, 24), (2, 2, 5, 66, 26), (1, 3, 4, 65, 28), (2, 1, 6, 2, 2), (1, 2, 3, 1024, 1024),
          (1, 70, 300, 128, 128), (5, 1, 257, 64, 32), (1, 7, 2, 256, 48), (1, 33, 1, 128, 4)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tin,tout", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,H,T,d,rot", SHAPES)
def test_rope(B, H, T, d, rot, tin, tout, layout):
    w = angles(rot)
    x, pos = rows((B, H, T, d), tin, 1, token_major=T % 2 == 1), positions(B, T, 2)
    ph = blkattn.rope_phases(w)
    y = blkattn.rope(x, pos, ph, layout=layout, mscale=1.25, out_dtype=tout)
    assert y.dtype == tout
    check(y, *turned(x, pos, w, layout, 1.25))
    dx = blkattn.rope_backward(x, pos, ph, layout=layout, mscale=1.25, out_dtype=tout)
    check(dx, *turned(x, pos, w, layout, 1.25, back=True))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_agrees_with_plain_angles(layout):
    # the reference above takes its angles from the phase table: at ordinary
    # positions it must be the rotation by pos * w (2^-53 pos of angle error)
    w = angles(64)
    x, pos = rows((2, 3, 50, 64), F32, 3), positions(2, 50, 4)
    y, _ = turned(x, pos, w, layout)
    a, b = pairs(64, layout)
    z = torch.complex(x.double().cpu()[..., a], x.double().cpu()[..., b])
    ang = pos.cpu().double()[:, None, :, None] * torch.tensor(w, dtype=torch.float64)
    z = z * torch.polar(torch.ones_like(ang), ang)
    torch.testing.assert_close(y[..., a], z.real, rtol=0, atol=1e-11)
    torch.testing.assert_close(y[..., b], z.imag, rtol=0, atol=1e-11)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    w = angles(128)
    x, pos = rows((2, 3, 64, 128), F32, 5), positions(2, 64, 6, far=True)
    check(blkattn.rope(x, pos, blkattn.rope_phases(w), layout=layout), *turned(x, pos, w, layout))


@pytest.mark.parametrize("d,rot,dtype", [(128, 128, BF16), (128, 64, BF16), (64, 24, F32), (66, 26, BF16)])
def test_in_place_is_the_same(d, rot, dtype):
    ph = blkattn.rope_phases(angles(rot))
    x, pos = rows((2, 5, 37, d), dtype, 7, token_major=True), positions(2, 37, 8)
    for f in (blkattn.rope, blkattn.rope_backward):
        want = f(x, pos, ph)
        y = x.clone(memory_format=torch.preserve_format)
        assert f(y, pos, ph, out=y) is y
        assert torch.equal(y, want)


def test_strided_broadcast_and_misaligned_views():
    ph, w = blkattn.rope_phases(angles(64)), angles(64)
    pos = positions(2, 19, 9)
    base = torch.randn(2, 4, 19, 200, generator=torch.Generator().manual_seed(10)).to(dev())
    for x in (base[..., 3:67], base[..., ::2][..., :64], base[:, :1, :, :64].expand(2, 4, 19, 64),
              base[:, :, :1, :64].expand(2, 4, 19, 64), base.to(BF16)[..., 1:65], base.to(BF16)[..., 8:72]):
        check(blkattn.rope(x, pos, ph), *turned(x, pos, w, "half"))
        out = torch.full((2, 4, 19, 131), 7.0, dtype=x.dtype, device=x.device)
        blkattn.rope(x, pos, ph, out=out[..., 2:66])
        check(out[..., 2:66], *turned(x, pos, w, "half"))
        assert bool((out[..., :2] == 7).all()) and bool((out[..., 66:] == 7).all())
    # positions and phases of other strides
    x = base[..., :64]
    pos2 = torch.zeros(19, 2, 2, dtype=torch.int32, device=dev())
    pos2[:, :, 0] = pos.t()
    ph2 = torch.zeros(32, 3, dtype=torch.int64, device=dev())
    ph2[:, 1] = ph
    assert torch.equal(blkattn.rope(x, pos2[:, :, 0].t(), ph2[:, 1]), blkattn.rope(x, pos, ph))
    one = pos[:1, :1].expand(2, 19)
    assert torch.equal(blkattn.rope(x, one, ph), blkattn.rope(x, one.contiguous(), ph))


def test_nonfinite_rows_stay_in_their_pairs():
    ph = blkattn.rope_phases(angles(64))
    x, pos = rows((1, 2, 5, 128), F32, 11), positions(1, 5, 12)
    clean = blkattn.rope(x, pos, ph)
    x[0, 1, 2, 7] = math.nan
    x[0, 0, 3, 100] = math.inf  # past the rotated dims: copied
    y = blkattn.rope(x, pos, ph)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1, 2, 7] = hit[0, 1, 2, 39] = True
    assert bool(y[hit].isnan().all())
    assert float(y[0, 0, 3, 100]) == math.inf
    hit[0, 0, 3, 100] = True
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_backward_is_the_transpose_and_the_difference(layout):
    # <dy, rope(x)> = <rope_bwd(dy), x> in 64 bits over f32 results: each
    # element within the bound above, so the two sums differ by at most
    # 2 * 6.2e-7 * mscale * sum |dy| (|x_a| + |x_b|)
    w, m = angles(48), 1.3
    ph = blkattn.rope_phases(w)
    x, dy, pos = rows((2, 3, 41, 64), F32, 13), rows((2, 3, 41, 64), F32, 14), positions(2, 41, 15)
    y, dx = blkattn.rope(x, pos, ph, layout=layout, mscale=m), blkattn.rope_backward(dy, pos, ph, layout=layout, mscale=m)
    lhs, rhs = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    ax, ay = x.double().abs(), dy.double().abs()
    bound = 2 * 6.2e-7 * m * float((ay.sum(-1) * ax.sum(-1)).sum())
    assert abs(float(lhs - rhs)) <= bound
    # differences: the map is linear, so one step along e_i gives column i
    # exactly up to the roundings of two results of size <= m (|x_a| + |x_b| + 1)
    L = dy.double()
    for b, h, t, i in ((0, 0, 0, 0), (1, 2, 40, 47), (0, 1, 7, 60), (1, 0, 3, 25)):
        e = torch.zeros_like(x)
        e[b, h, t, i] = 1.0
        d = ((blkattn.rope(x + e, pos, ph, layout=layout, mscale=m).double() - y.double()) * L)[b, h, t].sum()
        row = x[b, h, t].double().abs()
        tol = 2 * m * float((L[b, h, t].abs() * (2 * row.max() + 1)).sum()) * (6.2e-7 + 2 ** -24)
        assert abs(float(d) - float(dx[b, h, t, i])) <= tol


def test_side_stream_and_graph():
    ph, w = blkattn.rope_phases(angles(128)), angles(128)
    x, pos = rows((2, 8, 65, 128), BF16, 16), positions(2, 65, 17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    blkattn.rope(x, pos, ph, out=y, stream=s)
    s.synchronize()
    check(y, *turned(x, pos, w, "half"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = blkattn.rope(x, pos, ph)
        z = blkattn.rope_backward(z, pos, ph, out_dtype=F32)
    x.copy_(rows((2, 8, 65, 128), BF16, 18))
    pos.copy_(positions(2, 65, 19))
    g.replay()
    torch.cuda.synchronize()
    # there and back: two roundings of the kernel's arithmetic and one bf16 store
    _, bound = turned(x, pos, w, "half")
    pair = bound / 6.2e-7  # |x_a| + |x_b| of each element's pair
    err = (z.double().cpu() - x.double().cpu()).abs()
    assert bool((err <= pair * (2 * 2 * 6.2e-7 + 2 * 2.0 ** -8)).all())


# ------------------------------------------------------------------ append
def pools(N, H, P, d, dtype, rows_major, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (N, P, H, d) if rows_major else (N, H, P, d)
    a, b = (torch.randn(shape, generator=g).to(dtype).to(dev()) for _ in range(2))
    return (a.transpose(1, 2), b.transpose(1, 2)) if rows_major else (a, b)


def table_of(lens, P, entries, N, seed):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(N, generator=g).to(torch.int32)
    t = torch.full((len(lens), entries), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // P)
        t[b, :k] = order[at:at + k]
        at += k
    assert at <= N
    return t.to(dev())


def expect_append(k, v, pos, table, kp, vp, w, layout, mscale):
    """Pools after the call, in 64 bits, and the bounds before the store (0: not written)."""
    kt, kb = turned(k, pos, w, layout, mscale)
    wk, wv = kp.double().cpu().clone(), vp.double().cpu().clone()
    bk = torch.zeros_like(wk)
    hit = torch.zeros(wk.shape, dtype=torch.bool)
    N, _, P, _ = kp.shape
    p, tb = pos.cpu(), table.cpu()
    for b in range(p.shape[0]):
        for i in range(p.shape[1]):
            t = int(p[b, i])
            if t < 0 or t // P >= tb.shape[1] or not 0 <= int(tb[b, t // P]) < N:
                continue
            pg = int(tb[b, t // P])
            wk[pg, :, t % P], bk[pg, :, t % P] = kt[b, :, i], kb[b, :, i]
            wv[pg, :, t % P] = v[b, :, i].double().cpu()
            hit[pg, :, t % P] = True
    return wk, wv, bk, hit


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,T,d,rot,P,rows_major", [
    (1, 1, 1, 1, 128, 128, 8, False), (3, 8, 2, 1, 128, 128, 16, False), (4, 4, 4, 5, 64, 64, 16, True),
    (2, 6, 3, 70, 128, 64, 32, True), (2, 0, 2, 33, 64, 0, 64, False), (3, 7, 1, 19, 80, 24, 8, True),
    (2, 2, 2, 130, 66, 26, 128, False), (2, 4, 2, 9, 128, 0, 256, True), (1, 2, 1, 3, 5, 4, 16, False)])
def test_append(B, Hq, Hkv, T, d, rot, P, rows_major, dtype, layout):
    w = angles(rot) if rot else []
    lens = [1 + (37 * b) % 61 for b in range(B)]
    entries = max(-(-(n + T) // P) for n in lens)
    N = sum(-(-(n + T) // P) for n in lens) + 2
    kp, vp = pools(N, Hkv, P, d, dtype, rows_major, 20)
    table = table_of([n + T for n in lens], P, entries, N, 21)
    pos = (torch.tensor(lens)[:, None] + torch.arange(T)).to(torch.int32)
    if T > 2:
        pos[B - 1, T - 1] = -1        # padding
        pos[0, 1] = -7
    pos = pos.to(dev())
    k, v = rows((B, Hkv, T, d), dtype, 22, True), rows((B, Hkv, T, d), dtype, 23, True)
    q = rows((B, Hq, T, d), dtype, 24, True) if Hq else None
    q_out = torch.full((B, Hq, T, d), 5.0, dtype=dtype, device=dev()) if Hq else None
    wk, wv, bk, hit = expect_append(k, v, pos, table, kp, vp, w, layout, 1.1 if w else 1.0)
    old_k = kp.clone()
    blkattn.paged_append(k, v, pos, table, kp, vp, phases=blkattn.rope_phases(w) if w else None, layout=layout,
                         mscale=1.1, q=q, q_out=q_out)
    check(torch.where(hit.to(dev()), kp, torch.zeros_like(kp)), torch.where(hit, wk, torch.zeros_like(wk)), bk)
    assert torch.equal(kp[~hit.to(dev())], old_k[~hit.to(dev())])  # nothing else is written
    assert torch.equal(vp.double().cpu(), wv)                       # v is copied bit for bit
    if Hq:
        wq, bq = turned(q, pos, w, layout, 1.1 if w else 1.0)
        live = (pos >= 0)[:, None, :, None].expand_as(q_out)
        check(torch.where(live, q_out, torch.zeros_like(q_out)), torch.where(live.cpu(), wq, torch.zeros_like(wq)), bq)
        assert bool((q_out[~live] == 5).all())


def test_append_skips_what_holds_no_page():
    B, H, T, d, P, N = 4, 2, 6, 64, 16, 5
    kp, vp = pools(N, H, P, d, BF16, False, 30)
    k0, v0 = kp.clone(), vp.clone()
    table = torch.tensor([[0, -1], [N, 1], [2 ** 31 - 1, -(2 ** 31)], [3, 2]], dtype=torch.int32, device=dev())
    pos = torch.tensor([[0, 15, 16, 31, 32, 2 ** 31 - 1], [0, 15, 16, 17, 31, 32], [0, 5, 15, 16, 30, 31],
                        [32, 33, 47, 1000, -1, -(2 ** 31)]], dtype=torch.int32, device=dev())
    k, v = rows((B, H, T, d), BF16, 31), rows((B, H, T, d), BF16, 32)
    q = rows((B, 4, T, d), BF16, 33)
    w = angles(64)
    wk, wv, bk, hit = expect_append(k, v, pos, table, kp, vp, w, "half", 1.0)
    assert int(hit.any(-1).any(1).sum()) == 5  # (0: rows 0, 15; 1: rows 0, 1, 15 of page 1)
    qo = blkattn.paged_append(k, v, pos, table, kp, vp, phases=blkattn.rope_phases(w), q=q)
    h = hit.to(dev())
    check(torch.where(h, kp, torch.zeros_like(kp)), torch.where(hit, wk, torch.zeros_like(wk)), bk)
    assert torch.equal(kp[~h], k0[~h]) and torch.equal(vp[~h], v0[~h])
    wq, bq = turned(q, pos, w, "half")
    live = (pos >= 0)[:, None, :, None].expand_as(qo)
    check(qo, torch.where(live.cpu(), wq, torch.zeros_like(wq)), bq)


def test_append_same_row_twice_keeps_one_of_them():
    kp, vp = pools(3, 2, 8, 128, BF16, False, 40)
    k, v = rows((1, 2, 2, 128), BF16, 41), rows((1, 2, 2, 128), BF16, 42)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=dev())
    pos = torch.full((1, 2), 9, dtype=torch.int32, device=dev())
    k0 = kp.clone()
    blkattn.paged_append(k, v, pos, table, kp, vp)
    assert bool(((kp[0, :, 1] == k[0, :, 0]) | (kp[0, :, 1] == k[0, :, 1])).all())
    assert bool(((vp[0, :, 1] == v[0, :, 0]) | (vp[0, :, 1] == v[0, :, 1])).all())
    kp[0, :, 1] = k0[0, :, 1]
    assert torch.equal(kp, k0)


def test_append_offsets_past_32_bits():
    # a pool of more than 2^32 bytes and 2^31 elements
    P, H, d = 256, 8, 128
    N = (1 << 31) // (P * H * d) + 3
    kp = torch.zeros((N, P, H, d), dtype=BF16, device=dev()).transpose(1, 2)
    vp = torch.zeros((N, H, P, d), dtype=BF16, device=dev())
    table = torch.tensor([[N - 1, 0]], dtype=torch.int32, device=dev())
    pos = torch.tensor([[255, 256, 3]], dtype=torch.int32, device=dev())
    k, v = rows((1, H, 3, d), BF16, 43, True), rows((1, H, 3, d), BF16, 44, True)
    w = angles(d)
    blkattn.paged_append(k, v, pos, table, kp, vp, phases=blkattn.rope_phases(w))
    want, bound = turned(k, pos, w, "half")
    for i, (pg, r) in enumerate(((N - 1, 255), (0, 0), (N - 1, 3))):
        check(kp[pg, :, r], want[0, :, i], bound[0, :, i])
        assert torch.equal(vp[pg, :, r], v[0, :, i])
    assert int((vp[N - 1] != 0).any(-1).any(0).sum()) == 2 and int((vp[0] != 0).any(-1).any(0).sum()) == 1
    assert int(torch.count_nonzero(vp[1:N - 1])) == 0


def test_append_of_very_many_heads():
    # more heads than grid rows: 3 x 22000
    H, d = 22000, 16
    k, v, q = (rows((1, H, 1, d), BF16, 70 + i, True) for i in range(3))
    kp, vp = pools(2, H, 8, d, BF16, False, 73)
    table = torch.tensor([[1]], dtype=torch.int32, device=dev())
    pos = torch.tensor([[5]], dtype=torch.int32, device=dev())
    w = angles(d)
    ph = blkattn.rope_phases(w)
    qo = blkattn.paged_append(k, v, pos, table, kp, vp, phases=ph, q=q)
    check(qo, *turned(q, pos, w, "half"))
    check(kp[1, :, 5], *(z[0, :, 0] for z in turned(k, pos, w, "half")))
    assert torch.equal(vp[1, :, 5], v[0, :, 0])


def test_append_q_in_place_and_graph():
    w = angles(128)
    ph = blkattn.rope_phases(w)
    kp, vp = pools(6, 2, 16, 128, BF16, True, 50)
    k, v = rows((2, 2, 1, 128), BF16, 51), rows((2, 2, 1, 128), BF16, 52)
    q = rows((2, 8, 1, 128), BF16, 53)
    table = torch.tensor([[4, 1], [0, 5]], dtype=torch.int32, device=dev())
    pos = torch.tensor([[3], [20]], dtype=torch.int32, device=dev())
    want = blkattn.rope(q, pos, ph)
    blkattn.paged_append(k, v, pos, table, kp, vp, phases=ph, q=q, q_out=q)
    assert torch.equal(q, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blkattn.paged_append(k, v, pos, table, kp, vp, phases=ph)
    for step in range(3):
        pos += 1
        k.copy_(rows((2, 2, 1, 128), BF16, 60 + step))
        g.replay()
    torch.cuda.synchronize()
    for i, t in ((0, 6), (1, 23)):
        check(kp[int(table[i, t // 16]), :, t % 16], *(z[i, :, 0] for z in turned(k, pos, w, "half")))
