"""Attention over the 8-bit paged cache on the GPU, against an explicit 64-bit
softmax over the numbers that the cache stands for, and the operators of the
8-bit cache run together.

Tolerance, derived from the kernels' arithmetic.  A score is a sum of d exact
products accumulated in fp32 and multiplied by two fp32 factors: off by at most
E = 2^-23 (d + 6) scale sum |q||k| in natural-log units, which is also the
relative error of its weight.  A weight is 2^x by an approximation of 2^-22, and
enters the value product as one f16 (2^-11) for a bf16 out or as two (2^-22)
for f32; below 2^-36 of the largest weight times scale it loses all of it.  Both
sums over n keys are fp32 (2^-23 a step).  With e = E + 2^-11 (f32: 2^-21)
+ 2^-21 + n 2^-23, out is off by at most 2 e sum p |v| / sum p, plus
n 2^-36 448 max (p 2^ev) / sum p; lse by E + 2^-21 + n 2^-23 and 2^-21 |lse|.
Heads of 128 with a bf16 out go to the tcgen05 kernel.  Its scores add the rest
of q below 2^-22 of the row's largest dim, scale 2^-22 max |q| sum |k| each, its
weights are f16 in four e4m3 pieces: 2^-11 and half a step of 2^-23 of the largest
weight times scale, in place of 2^-36 (here 2^-24).
Prompts that go through the bf16 kernel have its bounds (test_gpu_paged.py):
2^-8 and 2^-16 in place of 2^-11.  A bf16 store adds 2^-8 of the value.
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_rotary import dev

pytestmark = pytest.mark.gpu
BF16, F32, F64, U8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def make(B, Hq, Hkv, Tq, d, P, S, lens, rows_major=False, seed=0, entries=None, sharp=1.0, spread=2, heads_first=False):
    """A problem whose pools and scales are NaN but for the rows [0, len) of each sequence (and their blocks'
    scales); entries past a sequence's pages are wild."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    N = sum(need) + 2
    entries = entries or max(1, max(need)) + 1
    order = torch.randperm(N, generator=g)
    table = torch.randint(-(2 ** 31), 2 ** 31, (B, entries), generator=g).to(I32)
    table[:, -1] = torch.randint(0, N, (B,), generator=g).to(I32)  # (some of them in range)
    shape = (N, P, Hkv, d) if rows_major else (N, Hkv, P, d)
    out = []
    for gain in (sharp, 1.0):
        pool = torch.full(shape, 0x7f, dtype=U8)
        if rows_major:
            pool = pool.transpose(1, 2)
        scales = torch.full((N, Hkv, P // S), 255, dtype=U8)
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = ids.to(I32)
            x = (torch.randn(Hkv, n, d, generator=g) * gain * 100).clamp(-448, 448).to(F8).view(U8)  # (past 464: NaN)
            e = torch.randint(-spread, spread + 1, (Hkv, -(-n // S)), generator=g) - 7
            for j, pg in enumerate(ids.tolist()):
                r = x[:, j * P:(j + 1) * P]
                pool[pg, :, :r.shape[1]] = r
                f = e[:, j * P // S:(j + 1) * P // S]
                scales[pg, :, :f.shape[1]] = (f + 127).to(U8)
        pool = pool.transpose(1, 2).contiguous().to(dev()).transpose(1, 2) if rows_major else pool.to(dev())
        out += [pool.view(F8), scales.to(dev()).view(E8)]
    q = torch.randn(B, Hq, Tq, d, generator=g) if heads_first else torch.randn(B, Tq, Hq, d, generator=g).transpose(1, 2)
    pos = torch.tensor([[n - Tq + i for i in range(Tq)] for n in lens], dtype=I32)
    return dict(q=q.to(BF16).to(dev()), kp=out[0], ks=out[1], vp=out[2], vs=out[3], table=table.to(dev()),
                lens=torch.tensor(lens, dtype=I32, device=dev()), pos=pos.to(dev()), scale=d ** -0.5, tree=None, window=0)


def call(a, out_dtype=F32, **kw):
    return blkattn.attention_paged_q8(a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["lens"], a["pos"],
                                      scale=a["scale"], out_dtype=out_dtype, tree=a["tree"], window=a["window"], **kw)


def reference(a, out_dtype):
    """(out, lse, out bound, lse bound but for the store), explicit and in 64 bits."""
    q = a["q"]
    B, Hq, Tq, d = q.shape
    N, Hkv, P, _ = a["kp"].shape
    S = P // a["ks"].shape[2]
    G = Hq // Hkv
    dv = q.device
    out = torch.zeros(B, Hq, Tq, d, dtype=F64, device=dv)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=F64, device=dv)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    table, lens, pos = a["table"].cpu(), a["lens"].cpu(), a["pos"].cpu()
    prompt = Tq >= 64 and a["tree"] is None and a["scale"] > 0 and q.stride(3) == 1 and q.stride(2) % 8 == 0
    wt = 2.0 ** -8 + 2.0 ** -16 if prompt else (2.0 ** -11 if out_dtype == BF16 else 2.0 ** -21)
    pieces = d == 128 and out_dtype == BF16 and not prompt and table.shape[1] * P > 256
    step = 2.0 ** -24 if pieces else 2.0 ** -36
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * P))
        ent = table[b, : -(-n // P)].long()
        ok = (ent >= 0) & (ent < N)
        has = ok.repeat_interleave(P)[:n].to(dv)
        j = torch.arange(n, device=dv)
        p = pos[b].long().to(dv)
        see = has[None] & (j[None] <= p[:, None])
        if a["window"]:
            see &= j[None] > (p - a["window"])[:, None]
        if a["tree"] is not None:
            node = (j - (n - Tq))[None]
            bits = (a["tree"][b][:, None] >> node.clamp(0, 63)) & 1
            see &= (node < 0) | (bits.bool() & (node < 64))
        if n == 0 or not bool(see.any()):
            continue
        used = see.any(0)[:, None]
        ids = ent.clamp(0, N - 1).masked_fill(~ok, 0).to(dv)
        for h in range(Hkv):
            kv = []
            for pool, scales in (("kp", "ks"), ("vp", "vs")):
                x = a[pool].view(U8)[ids, h].view(F8).double()
                e = a[scales].view(U8)[ids, h].double() - 127
                f = torch.exp2(e.masked_fill(e == 128, 0)).repeat_interleave(S, 1)[..., None]
                kv += [torch.where(used, (x * f).reshape(-1, d)[:n], 0.0), f.reshape(-1)[:n]]
            k, _, v, fv = kv
            z = torch.einsum("gtd,nd->gtn", q[b, h * G:(h + 1) * G].double(), k) * a["scale"]
            E = torch.einsum("gtd,nd->gtn", q[b, h * G:(h + 1) * G].double().abs(), k.abs()) * abs(a["scale"])
            E = E * 2.0 ** -23 * (d + 6)
            if pieces:
                top = q[b, h * G:(h + 1) * G].double().abs().amax(-1, keepdim=True)
                E = E + 2.0 ** -22 * abs(a["scale"]) * top * k.abs().sum(-1)
            E = E.masked_fill(~see, 0.0).amax(-1)
            z = z.masked_fill(~see, -math.inf)
            m = z.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(z - m)
            l = w.sum(-1, keepdim=True)
            l1 = torch.where(l > 0, l, 1.0)
            out[b, h * G:(h + 1) * G] = torch.where(l > 0, w @ v / l1, 0.0)
            e = E + wt + 2.0 ** -21 + n * 2.0 ** -23
            lost = n * step * 448 * (w * fv).amax(-1, keepdim=True) / l1
            ob[b, h * G:(h + 1) * G] = 2 * e[..., None] * (w @ v.abs() / l1) + torch.where(l > 0, lost, 0.0)
            s = (m + torch.log(l))[..., 0]
            lse[b, h * G:(h + 1) * G] = s
            lb[b, h * G:(h + 1) * G] = (E + (2.0 ** -16 if prompt else 0) + 2.0 ** -21 + n * 2.0 ** -23
                                        + torch.where(s == -math.inf, 0.0, s.abs()) * 2.0 ** -21)
    return out, lse, ob, lb


def check(a, got, out_dtype=F32):
    out, lse = got
    assert blkattn.check_device_error() == 0
    wo, wl, ob, lb = reference(a, out_dtype)
    none = wl == -math.inf
    assert torch.equal(lse == -math.inf, none)
    assert bool((out[none] == 0).all())
    tol = ob * (1 + 2.0 ** -8) + 2.0 ** -8 * wo.abs() if out_dtype == BF16 else ob + 2.0 ** -23 * wo.abs()
    err = (out.double() - wo).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())
    err = torch.where(none, 0.0, (lse.double() - wl).abs())
    assert bool((err <= lb).all()), float((err / lb.clamp(min=1e-30)).max())


def chain(T):
    return [(1 << (i + 1)) - 1 for i in range(T)]


CASES = [
    dict(B=1, Hq=1, Hkv=1, Tq=1, d=64, P=8, S=8, lens=[1]),
    dict(B=4, Hq=8, Hkv=2, Tq=1, d=128, P=16, S=16, lens=[1, 17, 300, 1000]),
    dict(B=3, Hq=16, Hkv=2, Tq=1, d=128, P=16, S=1, lens=[0, 5, 2047], rows_major=True),
    dict(B=2, Hq=3, Hkv=3, Tq=1, d=64, P=32, S=4, lens=[33, 700]),
    dict(B=2, Hq=7, Hkv=1, Tq=2, d=64, P=8, S=2, lens=[90, 1500], rows_major=True),
    dict(B=2, Hq=16, Hkv=2, Tq=5, d=128, P=32, S=32, lens=[129, 1111]),
    dict(B=1, Hq=8, Hkv=1, Tq=17, d=128, P=64, S=16, lens=[4000]),
    dict(B=1, Hq=4, Hkv=1, Tq=1, d=128, P=128, S=128, lens=[20011], sharp=3.0),
    dict(B=1, Hq=2, Hkv=1, Tq=1, d=128, P=256, S=64, lens=[5000], spread=40),
    dict(B=40, Hq=2, Hkv=1, Tq=1, d=64, P=16, S=8, lens=list(range(0, 400, 10))),
    dict(B=2, Hq=4, Hkv=2, Tq=70, d=128, P=16, S=16, lens=[70, 500], heads_first=True),
    dict(B=1, Hq=2, Hkv=1, Tq=130, d=64, P=8, S=1, lens=[900], rows_major=True),
    dict(B=2, Hq=2, Hkv=2, Tq=300, d=128, P=64, S=32, lens=[1000, 300]),
]


def ident(c):
    return "-".join("x".join(map(str, v[:4])) if isinstance(v, list) else str(v) for v in c.values())


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("case", CASES, ids=ident)
def test_causal(case, out):
    a = make(**case)
    check(a, call(a, out), out)


@pytest.mark.parametrize("window", [1, 16, 100, 5000])
@pytest.mark.parametrize("case", CASES[1:9] + CASES[10:], ids=ident)
def test_window(case, window):
    a = make(**case, seed=1)
    a["window"] = window
    if window == 100:  # pages that the window left behind are given back
        P = a["kp"].shape[2]
        for b, n in enumerate(case["lens"]):
            gone = max(0, n - case["Tq"] - window + 1) // P
            a["table"][b, :gone] = -1
    check(a, call(a, BF16), BF16)


@pytest.mark.parametrize("T,masks", [(1, [1]), (6, [1, 3, 5, 11, 19, 37]), (9, chain(9)), (64, chain(64)),
                                     (5, [0, 2, 4, 0, 16])])
def test_tree(T, masks):
    a = make(3, 8, 2, T, 128, 16, 8, [T, 200 + T, 1501])
    a["pos"][:] = a["lens"][:, None] - 1
    if T == 6:
        a["pos"][1, 4:] = -1
    masks = [m - (1 << 64) if m >= 1 << 63 else m for m in masks]
    a["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev()).expand(3, T).contiguous()
    if T == 5:  # nodes 0 and 3 are listed by no row: theirs may hold anything
        for b in range(3):
            for node in (0, 3):
                key = int(a["lens"][b]) - 5 + node
                page = int(a["table"][b, key // 16])
                a["vp"].view(U8)[page, :, key % 16] = 0x7f
                a["kp"].view(U8)[page, :, key % 16] = 0xff
    check(a, call(a, BF16), BF16)
    if T == 9:
        b = dict(a, tree=None, pos=(a["lens"][:, None] - 9 + torch.arange(9, device=dev())).to(I32))
        for x, y in zip(call(a), call(b)):
            assert torch.equal(x, y)  # a chain is ordinary verification


def test_rows_that_see_nothing():
    a = make(4, 8, 2, 3, 128, 16, 16, [50, 0, 300, 40])
    a["pos"][0, 1] = -1
    a["pos"][2] = -5
    a["table"][3, :] = -1
    check(a, call(a))
    a["pos"][:] = -1
    out, lse = call(a, BF16)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_missing_pages_and_long_lengths():
    a = make(2, 8, 2, 2, 128, 16, 8, [500, 640], entries=40)
    a["table"][0, 3] = -1
    a["table"][0, 20:25] = 2 ** 31 - 1
    a["table"][1, 0] = -7
    a["lens"][1] = 2 ** 31 - 1  # clamped to the table
    a["pos"][1] = 639
    check(a, call(a))


def test_scales_far_apart():
    """Blocks whose scales differ by 2^60: weights go by weight times scale, each row's own."""
    a = make(1, 4, 1, 1, 128, 16, 16, [160], spread=0)
    a["vs"].view(U8)[int(a["table"][0, 3])] = 180
    a["ks"].view(U8)[int(a["table"][0, 3])] = 90  # (scores of 0: the other keys' weights may vanish beside it)
    check(a, call(a))
    a["vs"].view(U8)[int(a["table"][0, 3])] = 60
    check(a, call(a))
    # a key that outweighs the rest, whose numbers are 2^-60 of theirs
    page = int(a["table"][0, 0])
    a["kp"].view(U8)[page, 0, 0] = a["q"][0, 0, 0].float().mul(100).to(F8).view(U8)
    a["ks"].view(U8)[page] = 127
    a["vs"].view(U8)[page] = 60
    check(a, call(a))


def test_rows_of_any_size():
    a = make(1, 8, 1, 2, 128, 16, 16, [200])
    size = torch.tensor([1, 1e-30, 1e-38, 0, 1e4, 300, 1e-5, 2.0 ** -133], device=dev())
    a["q"] = (a["q"].float() * size[None, :, None, None]).to(BF16)
    check(a, call(a))
    for s in (0.0, -0.3):
        a["scale"] = s
        check(a, call(a))


def test_nan_stays_in_its_rows():
    a = make(1, 8, 1, 2, 128, 16, 16, [300])
    clean = call(a)
    a["q"][0, 3, 1, 7] = math.nan
    out, lse = call(a)
    assert bool(out[0, 3, 1].isnan().all()) and bool(lse[0, 3, 1].isnan())
    for x, y in zip((out, lse), clean):
        x[0, 3, 1] = y[0, 3, 1]
        assert torch.equal(x, y)
    # a NaN key: the rows that see it (the second of each head)
    a = make(1, 8, 1, 2, 128, 16, 16, [300])
    page = int(a["table"][0, 299 // 16])
    a["kp"].view(U8)[page, 0, 299 % 16, 5] = 0x7f
    out, lse = call(a)
    assert bool(out[0, :, 1].isnan().all()) and bool(lse[0, :, 1].isnan().all())
    assert torch.equal(out[0, :, 0], clean[0][0, :, 0]) and torch.equal(lse[0, :, 0], clean[1][0, :, 0])


@pytest.mark.parametrize("out", [F32, BF16])
def test_layouts_of_rows_and_outputs(out):
    a = make(2, 8, 2, 3, 64, 16, 4, [77, 400])
    want = call(a, out)
    wide = torch.zeros(2, 3, 8, 128, dtype=BF16, device=dev())
    wide[..., ::2] = a["q"].transpose(1, 2)
    a["q"] = wide[..., ::2].transpose(1, 2)  # (a dim stride of 2)
    o = torch.full((3, 2, 8, 80), 7.0, dtype=out, device=dev())
    lse = torch.full((3, 8, 2), 7.0, device=dev())
    view = o.permute(1, 2, 0, 3)[..., :64]
    blkattn.fwd_paged_q8(a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["lens"], a["pos"], a["scale"], view,
                         lse.permute(2, 1, 0))
    assert torch.equal(view, want[0]) and torch.equal(lse.permute(2, 1, 0), want[1]) and bool((o[..., 64:] == 7).all())


def test_strided_prompt():
    """Prompt rows that the prompt kernel does not take."""
    a = make(1, 2, 1, 80, 64, 16, 16, [300])
    wide = torch.zeros(1, 80, 2, 128, dtype=BF16, device=dev())
    wide[..., ::2] = a["q"].transpose(1, 2)
    a["q"] = wide[..., ::2].transpose(1, 2)
    check(a, call(a, BF16), BF16)


def test_batch_longer_than_a_launch():
    lens = [(i * 37) % 90 for i in range(800)]
    a = make(800, 2, 1, 1, 64, 8, 8, lens)
    check(a, call(a))


def test_pages_far_into_the_pool():
    """Page offsets past 2^31 bytes."""
    P, d, N = 256, 128, 70000
    pools = [torch.zeros(N, 1, P, d, dtype=U8, device=dev()) for _ in range(2)]
    scales = [torch.full((N, 1, 1 + 1), 127, dtype=U8, device=dev()) for _ in range(2)]
    a = make(1, 4, 1, 1, d, P, 128, [1000])
    ids = torch.tensor([N - 1, 5, N - 3, N - 2], device=dev())
    for i, n in enumerate(("kp", "vp")):
        pools[i][ids] = a[n].view(U8)[a["table"][0, :4].long()]
    for i, n in enumerate(("ks", "vs")):
        scales[i][ids] = a[n].view(U8)[a["table"][0, :4].long()]
    want = call(a)
    b = dict(a, kp=pools[0].view(F8), vp=pools[1].view(F8), ks=scales[0].view(E8), vs=scales[1].view(E8),
             table=ids.to(I32)[None].contiguous())
    a["table"] = a["table"][:, :4].contiguous()
    for x, y in zip(call(b), call(a)):
        assert torch.equal(x, y)
    check(a, call(b))
    assert want[0].shape == (1, 4, 1, d)


def test_captured_calls_share_the_workspace():
    a = make(3, 8, 2, 2, 128, 16, 16, [900, 100, 2000])
    b = make(1, 16, 2, 1, 64, 32, 8, [5000], seed=5)
    c = make(1, 2, 1, 70, 128, 16, 16, [300], seed=6)
    want = [t.clone() for x in (a, b, c) for t in call(x)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs += call(x)
        graphs.append(g)
    for order in ((0, 1, 2), (2, 1, 0), (1, 1, 0, 2, 0)):
        for t in outs:
            t.fill_(7)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("d,P,S", [(128, 16, 16), (64, 32, 8)])
def test_a_serving_run(d, P, S):
    """A prompt in two chunks, then decode steps: norm, rotation and append, then attention, with the whole of it in
    64 bits from the numbers that the cache holds."""
    B, Hq, Hkv, T = 2, 8, 2, 96
    g = torch.Generator().manual_seed(3)
    N = 2 * 10
    kp, vp = (torch.full((N, Hkv, P, d), 0x7f, dtype=U8, device=dev()).view(F8) for _ in range(2))
    ks, vs = (torch.full((N, Hkv, P // S), 255, dtype=U8, device=dev()).view(E8) for _ in range(2))
    table = torch.randperm(N, generator=g).to(I32).reshape(B, 10).to(dev())
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(BF16).to(dev()) for _ in range(2))
    ph = blkattn.rope_phases(blkattn.rope_angles(d)[0])
    done = [0, 0]
    for step, news in enumerate(([96, 70], [37, 64], [1, 1], [1, 1], [5, 3])):
        n = max(news)
        pos = torch.full((B, n), -1, dtype=I32)
        for b in range(B):
            pos[b, :news[b]] = torch.arange(done[b], done[b] + news[b])
            done[b] += news[b]
        pos = pos.to(dev())
        k, v, q = (torch.randn(B, n, h, d, generator=g).to(BF16).to(dev()).transpose(1, 2) for h in (Hkv, Hkv, Hq))
        q = blkattn.paged_append_q8(k, v, pos, table, kp, vp, ks, vs, phases=ph, k_weight=wk, q_weight=wq, q=q)
        want_q, _ = blkattn.qk_norm_rope(k, None, wk, None, pos, ph, out_dtype=F32)
        back, _ = blkattn.paged_read_q8(pos, table, kp, vp, ks, vs, out_dtype=F32)
        live = (pos >= 0)[:, None, :, None]
        # what was written stands for the normed, turned rows: half a step of e4m3, 2^-4 of the value or 2^-10 2^e
        # (2^e <= amax / 224), and both norms' fp32 errors
        bound = 2.0 ** -4 * want_q.abs() + (2.0 ** -17 + 2.0 ** -18) * want_q.abs().amax()
        assert bool(((back - want_q).abs() <= bound)[live.expand_as(back)].all())
        a = dict(q=q, kp=kp, vp=vp, ks=ks, vs=vs, table=table, lens=torch.tensor(done, dtype=I32, device=dev()), pos=pos,
                 scale=d ** -0.5, tree=None, window=0)
        check(a, call(a, BF16), BF16)
