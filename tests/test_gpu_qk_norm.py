"""Head norms with rotation and their gradients on the GPU, against 64 bits.

Tolerance, derived from the kernels' arithmetic.  The sum of d squares is off by
d 2^-24 of itself, half of that through the root, which adds 2 units (2^-22);
the products with r and w add two roundings: the normed row is off by at most
N = (d / 2 + 8) 2^-24 + 2^-22 of itself.  The rotation adds 6.2e-7 mscale
(|u_a| + |u_b|) (test_gpu_rotary.py), the store half a step of the value.

Gradient: g = R^T dy is off by A = 6.2e-7 of G = mscale (|dy_a| + |dy_b|), the
root by N, a sum of d products by d 2^-24 of the sum of their sizes, the last
expression by four roundings: dx by at most
(A + 3 N + (d + 8) 2^-24) r (C + |h| mean(C |h|)), C = |w| G.  A sum of n rows
adds at most n roundings: dw by (A + N + (n + 4) 2^-24) sum G |h|.
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_rotary import angles, check, dev, pairs, turned

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def problem(B, Hq, Hk, T, d, rot, dtype=BF16, first=0, seed=0, view=None, wtype=BF16):
    """q, k as token-major views (or contiguous, or with a dim stride), weights, positions, angles."""
    g = torch.Generator().manual_seed(seed)

    def rows(H):
        x = torch.randn(B, T, H, d, generator=g) * torch.exp(torch.randn(B, T, H, 1, generator=g))
        x = x.to(dtype).to(dev())
        if view == "contiguous":
            return x.transpose(1, 2).contiguous()
        if view == "strided":  # every second dim of a wider row
            wide = torch.zeros(B, T, H, 2 * d, dtype=dtype, device=dev())
            wide[..., ::2] = x
            return wide[..., ::2].transpose(1, 2)
        return x.transpose(1, 2)

    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(wtype).to(dev()) for _ in range(2)]
    pos = (torch.randint(0, first + 1, (B, 1), generator=g) + torch.arange(T)).to(torch.int32).to(dev())
    return rows(Hq), rows(Hk), *w, pos, angles(rot) if rot else []


def normed(x, w):
    x, w = x.double().cpu(), w.double().cpu()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def n_of(d):
    return (d / 2 + 8) * 2.0 ** -24 + 2.0 ** -22


def check_forward(got, x, w, pos, ang, layout, mscale):
    u = normed(x, w)
    want, bound = turned(u, pos, ang, layout, mscale)
    size = u.abs()
    if ang:
        a, b = pairs(2 * len(ang), layout)
        size[..., a] = size[..., b] = abs(mscale) * (u[..., a].abs() + u[..., b].abs())
    check(got, want, bound + n_of(x.shape[-1]) * size)


CASES = [
    dict(B=3, Hq=4, Hk=2, T=1, d=128, rot=128),
    dict(B=2, Hq=5, Hk=3, T=70, d=128, rot=128, layout="interleaved", first=1000000),
    dict(B=1, Hq=33, Hk=1, T=9, d=64, rot=64, mscale=1.2),
    dict(B=2, Hq=3, Hk=3, T=17, d=64, rot=24, layout="interleaved", dtype=F32),
    dict(B=2, Hq=3, Hk=2, T=17, d=64, rot=22, dtype=F32, out=BF16),
    dict(B=1, Hq=2, Hk=2, T=19, d=128, rot=64, dtype=F32, view="contiguous"),
    dict(B=2, Hq=2, Hk=1, T=11, d=128, rot=32, view="strided", wtype=F32),
    dict(B=2, Hq=4, Hk=4, T=8, d=96, rot=96, out=F32),
    dict(B=1, Hq=2, Hk=1, T=5, d=7, rot=6, dtype=F32),
    dict(B=1, Hq=1, Hk=1, T=3, d=1024, rot=1024),
    dict(B=2, Hq=2, Hk=2, T=6, d=256, rot=0),
    dict(B=1, Hq=2, Hk=2, T=6, d=48, rot=0, dtype=F32),
]


def ident(c):
    return "-".join(str(v).replace("torch.", "") for v in c.values())


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_forward(case):
    c = dict(case)
    layout, mscale, out = c.pop("layout", "half"), c.pop("mscale", 1.0), c.pop("out", None)
    q, k, wq, wk, pos, ang = problem(**c)
    ph = blkattn.rope_phases(ang) if ang else None
    kw = dict(eps=EPS, layout=layout, mscale=mscale)
    qo, ko = blkattn.qk_norm_rope(q, k, wq, wk, pos, ph, out_dtype=out, **kw)
    assert qo.dtype == (out or q.dtype) and qo.shape == q.shape and ko.shape == k.shape
    check_forward(qo, q, wq, pos, ang, layout, mscale)
    check_forward(ko, k, wk, pos, ang, layout, mscale)
    # one set alone, and outputs given in an order of their own
    q1 = torch.full((q.shape[2], q.shape[0], q.shape[1], q.shape[3] + 8), 7.0, dtype=qo.dtype, device=dev())
    view = q1.permute(1, 2, 0, 3)[..., :q.shape[3]]
    got, none = blkattn.qk_norm_rope(q, None, wq, None, pos, ph, q_out=view, **kw)
    assert got is view and none is None and bool((q1[..., q.shape[3]:] == 7).all())
    check_forward(view, q, wq, pos, ang, layout, mscale)
    if out is None:  # in place
        q2, k2 = q.clone(), k.clone()
        blkattn.qk_norm_rope(q2, k2, wq, wk, pos, ph, q_out=q2, k_out=k2, **kw)
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


def exact_gradient(dy, x, w, pos, ang, layout, mscale):
    """(dx, bound, dw, bound) of the formula."""
    g, bg = turned(dy, pos, ang, layout, mscale, back=True)
    d = x.shape[-1]
    dyc = dy.double().cpu()
    G = dyc.abs()
    if ang:
        a, b = pairs(2 * len(ang), layout)
        G[..., a] = G[..., b] = abs(mscale) * (dyc[..., a].abs() + dyc[..., b].abs())
    x, w = x.double().cpu(), w.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    h, c, C = x * r, w * g, w.abs() * G
    dx = r * (c - h * (c * h).mean(-1, keepdim=True))
    A, N = 6.2e-7, n_of(d)
    bx = (A + 3 * N + (d + 8) * 2.0 ** -24) * r * (C + h.abs() * (C * h.abs()).mean(-1, keepdim=True))
    n = x.shape[0] * x.shape[1] * x.shape[2]
    return dx, bx, (g * h).sum((0, 1, 2)), (A + N + (n + 4) * 2.0 ** -24) * (G * h.abs()).sum((0, 1, 2))


@pytest.mark.parametrize("gtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES, ids=ident)
def test_gradient(case, gtype):
    c = dict(case)
    layout, mscale, out = c.pop("layout", "half"), c.pop("mscale", 1.0), c.pop("out", None)
    q, k, wq, wk, pos, ang = problem(**c, seed=3)
    ph = blkattn.rope_phases(ang) if ang else None
    g = torch.Generator().manual_seed(9)
    gq, gk = (torch.randn(x.shape, generator=g).to(gtype).to(dev()) for x in (q, k))
    kw = dict(eps=EPS, layout=layout, mscale=mscale, out_dtype=out)
    dq, dk, dwq, dwk = blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph, **kw)
    for dx, dw, dy, x, w in ((dq, dwq, gq, q, wq), (dk, dwk, gk, k, wk)):
        wx, bx, ww, bw = exact_gradient(dy, x, w, pos, ang, layout, mscale)
        check(dx, wx, bx)
        assert dw.dtype == F32
        check(dw, ww, bw)
    again = blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))
    one = blkattn.qk_norm_rope_backward(gq, None, q, None, wq, None, pos, ph, **kw)
    assert torch.equal(one[0], dq) and one[1] is None and one[3] is None
    check(one[2], *exact_gradient(gq, q, wq, pos, ang, layout, mscale)[2:])


def test_gradient_of_many_rows():
    """More tokens than one sweep of the grid, and gradients as views."""
    q, k, wq, wk, pos, ang = problem(2, 9, 2, 3000, 128, 128, seed=5)
    ph = blkattn.rope_phases(ang)
    gq = torch.randn(2, 3000, 9, 128, device=dev()).transpose(1, 2)
    gk = torch.randn(2, 2, 3000, 128, device=dev())
    dq, dk, dwq, dwk = blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph, eps=EPS)
    for dx, dw, dy, x, w in ((dq, dwq, gq, q, wq), (dk, dwk, gk, k, wk)):
        wx, bx, ww, bw = exact_gradient(dy, x, w, pos, ang, "half", 1.0)
        check(dx, wx, bx)
        check(dw, ww, bw)


def test_gradient_against_differences():
    """Central differences of L = sum dy . y in 64 bits.  With a step s their error is s^2 / 6 times a third
    derivative of L, here below 1e3 sum |dy| (rows of size 1, s = 1e-4), and 2^-52 L / s of rounding."""
    q, k, wq, wk, pos, ang = problem(1, 2, 1, 2, 16, 8, dtype=F32, seed=7)
    ph = blkattn.rope_phases(ang)
    gq, gk = (torch.randn(x.shape, device=dev()) for x in (q, k))
    dq, _, dwq, _ = blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph, eps=EPS)
    x, w, dy, s = q.double().cpu(), wq.double().cpu(), gq.double().cpu(), 1e-4

    def loss(x, w):
        return float((turned(normed(x, w), pos, ang, "half")[0] * dy).sum())

    def difference(of, which):
        grad = torch.zeros(of.numel(), dtype=F64)
        for i in range(of.numel()):
            e = torch.zeros(of.numel(), dtype=F64)
            e[i] = s
            e = e.reshape(of.shape)
            up, down = ((x + e, w), (x - e, w)) if which == 0 else ((x, w + e), (x, w - e))
            grad[i] = (loss(*up) - loss(*down)) / (2 * s)
        return grad.reshape(of.shape)

    _, bx, _, bw = exact_gradient(gq, q, wq, pos, ang, "half", 1.0)
    slack = s * s / 6 * 1e3 * float(dy.abs().sum()) + 2.0 ** -52 * abs(loss(x, w)) / s * 10
    check(dq, difference(x, 0), bx + slack)
    check(dwq, difference(w, 1), bw + slack)


def test_no_rows_and_empty_sets():
    q, k, wq, wk, pos, ang = problem(2, 3, 2, 4, 64, 64)
    ph = blkattn.rope_phases(ang)
    qo, ko = blkattn.qk_norm_rope(q[:, :0], k, wq, wk, pos, ph)
    assert qo.shape[1] == 0 and torch.equal(ko, blkattn.qk_norm_rope(k, None, wk, None, pos, ph)[0])
    qo, ko = blkattn.qk_norm_rope(q, k[:, :0], wq, wk, pos, ph)
    assert ko.shape[1] == 0 and torch.equal(qo, blkattn.qk_norm_rope(q, None, wq, None, pos, ph)[0])
    for x, y, p in ((q[:, :, :0], k[:, :, :0], pos[:, :0]), (q[:0], k[:0], pos[:0]), (q[:, :0], k[:, :0], pos)):
        grads = blkattn.qk_norm_rope_backward(x.float(), y.float(), x, y, wq, wk, p, ph)
        assert grads[0].shape == x.shape and bool((grads[2] == 0).all()) and bool((grads[3] == 0).all())


def test_a_bad_row_stays_its_own():
    """NaN, infinities and zeros in one row do not reach another row's result."""
    q, k, wq, wk, pos, ang = problem(1, 4, 1, 16, 128, 128)
    ph = blkattn.rope_phases(ang)
    clean, _ = blkattn.qk_norm_rope(q, None, wq, None, pos, ph)
    bad = q.clone()
    bad[0, 1, 3, 5] = math.nan
    bad[0, 2, 3, 64] = math.inf
    bad[0, 3, 3] = 0
    got, _ = blkattn.qk_norm_rope(bad, None, wq, None, pos, ph)
    assert bool(got[0, 1, 3].isnan().all()) and bool(got[0, 2, 3].isnan().any()) and bool((got[0, 3, 3] == 0).all())
    got[0, 1:, 3] = clean[0, 1:, 3]
    assert torch.equal(got, clean)


def test_captured_and_replayed():
    q, k, wq, wk, pos, ang = problem(2, 8, 2, 40, 128, 128)
    ph = blkattn.rope_phases(ang)
    gq, gk = (torch.randn(x.shape, device=dev()) for x in (q, k))
    want = blkattn.qk_norm_rope(q, k, wq, wk, pos, ph) + blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blkattn.qk_norm_rope(q, k, wq, wk, pos, ph) + blkattn.qk_norm_rope_backward(gq, gk, q, k, wq, wk, pos, ph)
    for _ in range(2):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
