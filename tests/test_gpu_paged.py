"""Attention over the paged cache on the GPU, against an explicit 64-bit
softmax, and the operators of the paged cache run together.

Tolerance, derived from the kernels' arithmetic.  A score is a sum of d fp32
products accumulated in fp32 (2^-23 a step, however the unit rounds): off by
at most E = 2^-23 (d + 4) scale sum |q||k| in natural-log units, which is also
the relative error of its weight.  A weight is 2^x by an approximation of
2^-22, carried as two bf16 (2^-16) or, on the prompt kernel's fully visible
tiles, as one (2^-8); n keys are summed in fp32 (2^-23 a step).  With
e = E + 2^-16 + 2^-21 + n 2^-23 (prompt kernel: + 2^-8) the quotient is off by
at most 2 e sum p |v| / sum p, and ln(sum p) by e plus its own roundings
(2^-21 |lse|).  A bf16 store adds 2^-8 of the value.
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def dev():
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def make(B, Hq, Hkv, Tq, d, P, lens, dtype=BF16, rows_major=False, seed=0, spare=2, entries=None, sharp=1.0,
         poison=True):
    """A problem whose pools are NaN but for the rows [0, len) of each
    sequence; entries past a sequence's pages are wild."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    N = sum(need) + spare
    entries = entries or max(1, max(need)) + 1
    order = torch.randperm(N, generator=g)
    table = torch.randint(-(2 ** 31), 2 ** 31, (B, entries), generator=g).to(torch.int32)
    table[:, -1] = torch.randint(0, N, (B,), generator=g).to(torch.int32)  # (some of them in range)
    shape = (N, P, Hkv, d) if rows_major else (N, Hkv, P, d)
    kp, vp = (torch.full(shape, math.nan if poison else 0.0, dtype=dtype) for _ in range(2))
    if rows_major:
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    at = 0
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids.to(torch.int32)
        for pool, gain in ((kp, sharp), (vp, 1.0)):
            x = (torch.randn(Hkv, n, d, generator=g) * gain).to(dtype)
            for j, pg in enumerate(ids.tolist()):
                r = x[:, j * P:(j + 1) * P]
                pool[pg, :, :r.shape[1]] = r
    q = torch.randn(B, Tq, Hq, d, generator=g).to(dtype).transpose(1, 2)
    pos = torch.tensor([[n - Tq + i for i in range(Tq)] for n in lens], dtype=torch.int32)
    to = dev()

    def up(t):
        return t.to(to)

    return dict(q=up(q), kp=up(kp.transpose(1, 2).contiguous()).transpose(1, 2) if rows_major else up(kp),
                vp=up(vp.transpose(1, 2).contiguous()).transpose(1, 2) if rows_major else up(vp), table=up(table),
                lens=up(torch.tensor(lens, dtype=torch.int32)), pos=up(pos), scale=d ** -0.5, tree=None, window=0)


def call(a, out_dtype=F32, **kw):
    return blkattn.attention_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["pos"], scale=a["scale"],
                                   out_dtype=out_dtype, tree=a["tree"], window=a["window"], **kw)


def reference(a):
    """(out, lse, out bound, lse bound but for the store), explicit and in 64 bits."""
    q, kp, vp = a["q"], a["kp"], a["vp"]
    B, Hq, Tq, d = q.shape
    N, Hkv, P, _ = kp.shape
    G = Hq // Hkv
    out = torch.zeros(B, Hq, Tq, d, dtype=F64, device=q.device)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=F64, device=q.device)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    table, lens, pos = a["table"].cpu(), a["lens"].cpu(), a["pos"].cpu()
    prompt = q.dtype == BF16 and Tq >= 64 and a["tree"] is None and a["scale"] > 0
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * P))
        ent = table[b, : -(-n // P)].long()
        ok = (ent >= 0) & (ent < N)
        has = ok.repeat_interleave(P)[:n].to(q.device)
        j = torch.arange(n, device=q.device)
        p = pos[b].long().to(q.device)
        see = has[None] & (j[None] <= p[:, None])
        if a["window"]:
            see &= j[None] > (p - a["window"])[:, None]
        if a["tree"] is not None:
            node = (j - (n - Tq))[None]
            bits = (a["tree"][b][:, None] >> node.clamp(0, 63)) & 1
            see &= (node < 0) | (bits.bool() & (node < 64))
        if n == 0 or not bool(see.any()):
            continue
        used = see.any(0)
        ids = ent.clamp(0, N - 1).masked_fill(~ok, 0).to(q.device)
        for h in range(Hkv):
            k = kp[ids, h].double().reshape(-1, d)[:n]
            v = vp[ids, h].double().reshape(-1, d)[:n]
            k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
            qq = q[b, h * G:(h + 1) * G].double()
            z = torch.einsum("gtd,nd->gtn", qq, k) * a["scale"]
            E = torch.einsum("gtd,nd->gtn", qq.abs(), k.abs()) * abs(a["scale"]) * 2.0 ** -23 * (d + 4)
            z = z.masked_fill(~see, -math.inf)
            E = E.masked_fill(~see, 0.0).amax(-1)
            m = z.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(z - m)
            l = w.sum(-1, keepdim=True)
            live = l > 0
            o = torch.where(live, w @ v / torch.where(live, l, 1.0), 0.0)
            av = torch.where(live, w @ v.abs() / torch.where(live, l, 1.0), 0.0)
            e = E + 2.0 ** -16 + 2.0 ** -21 + n * 2.0 ** -23 + (2.0 ** -8 if prompt else 0.0)
            out[b, h * G:(h + 1) * G], ob[b, h * G:(h + 1) * G] = o, 2 * e[..., None] * av
            s = (m + torch.log(l))[..., 0]
            lse[b, h * G:(h + 1) * G] = s
            lb[b, h * G:(h + 1) * G] = e + 2.0 ** -21 * torch.where(live[..., 0], s.abs(), 0.0)
    return out, lse, ob, lb


def check(a, out, lse):
    assert blkattn.check_device_error() == 0
    ro, rl, ob, lb = reference(a)
    empty = rl == -math.inf
    assert bool((out[empty].float() == 0).all()) and bool((lse[empty] == -math.inf).all())
    assert not bool(torch.signbit(out[empty].float()).any())
    tol = ob * (1 + 2.0 ** -8) + (2.0 ** -8 * ro.abs() if out.dtype == BF16 else 2.0 ** -24 * ro.abs())
    err = (out.double() - ro).abs()
    assert bool(torch.isfinite(out.float()).all())
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol.clamp_min(1e-30)).max()))
    le = (lse.double() - rl).abs()[~empty]
    assert bool((le <= lb[~empty]).all()), float((le - lb[~empty]).max())


DECODE = [
    # B, Hq, Hkv, Tq, d, P, lens
    (1, 1, 1, 1, 128, 16, [1]), (1, 4, 1, 1, 64, 8, [7]), (2, 8, 2, 1, 128, 8, [128, 129]),
    (3, 8, 2, 1, 64, 16, [1000, 0, 333]), (4, 32, 8, 1, 128, 16, [511, 1, 2050, 127]),
    (2, 14, 2, 2, 128, 32, [640, 77]), (1, 64, 8, 5, 128, 64, [3001]), (2, 64, 8, 5, 64, 128, [1285, 300]),
    (1, 16, 2, 17, 128, 256, [1500]), (2, 6, 3, 9, 64, 512, [513, 700]), (1, 2, 2, 33, 64, 16, [50]),
    (1, 1, 1, 100, 64, 32, [400]), (5, 7, 1, 3, 128, 16, [3, 4, 5, 255, 256]), (1, 3, 3, 63, 128, 8, [63]),
]


@pytest.mark.parametrize("rows_major", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,d,P,lens", DECODE)
def test_decode_and_verify(B, Hq, Hkv, Tq, d, P, lens, dtype, out_dtype, rows_major):
    a = make(B, Hq, Hkv, Tq, d, P, lens, dtype, rows_major, seed=Tq + d)
    check(a, *call(a, out_dtype))


PROMPT = [(1, 2, 1, 64, 16, [64]), (2, 4, 2, 130, 8, [130, 700]), (1, 4, 1, 300, 64, [1111]),
          (2, 2, 2, 257, 128, [257, 2000]), (1, 8, 2, 511, 256, [600]), (1, 1, 1, 1000, 32, [1000])]


@pytest.mark.parametrize("rows_major", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,P,lens", PROMPT)
def test_prompt_chunks(B, Hq, Hkv, Tq, P, lens, d, out_dtype, rows_major):
    a = make(B, Hq, Hkv, Tq, d, P, lens, BF16, rows_major, seed=Tq)
    check(a, *call(a, out_dtype))


@pytest.mark.parametrize("Hq,Hkv,Tq,d,K,window", [(4, 1, 64, 128, 9000, 0), (1, 1, 130, 128, 8200, 0),
                                                  (4, 4, 200, 128, 8192, 0), (8, 1, 100, 64, 6000, 0),
                                                  (1, 1, 300, 128, 8000, 3000), (2, 1, 2, 64, 40000, 0)])
def test_few_rows_over_long_contexts(Hq, Hkv, Tq, d, K, window):
    # prompt rows that the decode kernel serves; units split over many CTAs
    a = make(1, Hq, Hkv, Tq, d, 32, [K], seed=Tq + K)
    a["window"] = window
    check(a, *call(a, BF16))


# fp32 rows above 8 per KV head: 9 to 140 of them, whole and split, even and odd
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,P,lens", [
    (1, 9, 1, 1, 16, [700]), (2, 8, 4, 8, 32, [500, 33]), (3, 4, 2, 9, 8, [0, 18, 90]), (1, 20, 2, 3, 64, [1500]),
    (2, 12, 3, 10, 16, [200, 4000]), (1, 47, 1, 1, 256, [300]), (1, 4, 1, 14, 16, [14]), (1, 8, 1, 8, 128, [9000]),
    (1, 5, 1, 13, 16, [900]), (2, 7, 1, 20, 32, [100, 1000]), (1, 1, 1, 333, 16, [1200]), (40, 8, 8, 17, 16, [260] * 40)])
def test_many_f32_rows(B, Hq, Hkv, Tq, P, lens, d):
    a = make(B, Hq, Hkv, Tq, d, P, lens, F32, rows_major=Tq % 2 == 0, seed=Tq + d)
    want = call(a)
    check(a, *want)
    check(a, *call(a, BF16))
    # query rows behind one another at an odd stride, and dims apart: the same bits
    for buf, view in ((torch.zeros(B, Tq, Hq, d + 3, device=dev()), lambda t: t[..., 2:d + 2].transpose(1, 2)),
                      (torch.zeros(B, Hq, d, Tq, device=dev()), lambda t: t.transpose(2, 3))):
        q = view(buf)
        q.copy_(a["q"])
        out, lse = call(dict(a, q=q))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [128, 64])
def test_many_f32_rows_with_windows_trees_and_missing_pages(d):
    a = make(2, 6, 2, 40, d, 16, [3000, 777], F32, seed=97)
    for window in (1, 50, 1000):
        a["window"] = window
        check(a, *call(a))
    a["window"] = 0
    a["pos"][0, 3:9] = -1
    a["pos"][1, 30:] += 100
    a["table"][0, 5] = -1
    a["table"][0, 60:100] = 1 << 30
    check(a, *call(a))
    a["q"][0, :, 3:9] = math.nan  # padding rows may hold anything
    out, lse = call(a)
    assert bool((out[0, :, 3:9] == 0).all()) and bool((lse[0, :, 3:9] == -math.inf).all())
    assert bool(torch.isfinite(out).all())


# prompts whose last items are cut into parts along their keys: fewer items than
# SMs, sequences much shorter than the table (parts without a key), one wave of
# items and a rest
PARTS = [(1, 4, 1, 100, 16, [3000]), (3, 4, 2, 300, 32, [2500, 310, 1300]), (1, 3, 3, 700, 256, [4001]),
         (2, 1, 1, 64, 8, [64, 9000]), (4, 40, 8, 64, 32, [4096, 100, 4000, 2049])]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,P,lens", PARTS)
def test_prompts_in_parts(B, Hq, Hkv, Tq, P, lens, d, out_dtype):
    a = make(B, Hq, Hkv, Tq, d, P, lens, seed=Tq + d)
    check(a, *call(a, out_dtype))


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [0, 1, 100, 2600, 1 << 20])
def test_prompts_in_parts_with_windows_and_edges(window, d):
    lens = [4100, 300, 2900]
    a = make(3, 2, 1, 270, d, 16, lens, seed=71)
    a["window"] = window
    for b, n in enumerate(lens):  # pages behind every window hold nothing
        gone = max(0, n - 270 - window + 1) // 16 if window else 0
        a["kp"][a["table"][b, :gone].long()] = math.nan
        a["vp"][a["table"][b, :gone].long()] = math.nan
        a["table"][b, :gone] = -1
    a["pos"][0, :100] = torch.arange(3000, 3100, dtype=torch.int32, device=dev())  # not in order of the keys
    if window:
        a["pos"][0, :100] = a["pos"][0, 100:200]
    a["pos"][1, 200:] = -1                     # padding rows
    a["pos"][2, :128] = -7                     # a whole row tile without keys
    a["pos"][2, 128:] += 10                    # and rows past the end
    check(a, *call(a, BF16))


@pytest.mark.parametrize("d", [128, 64])
def test_prompts_in_parts_without_some_pages(d):
    a = make(2, 3, 1, 140, d, 32, [3500, 2000], seed=73)
    a["table"][0, 3] = -1
    a["table"][0, 40:70] = 1 << 30             # whole parts
    a["table"][1, 62] = -5                     # the last keys
    check(a, *call(a, F32))


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("d,window", [(128, 0), (64, 0), (128, 3000), (64, 3000)])
def test_prompts_in_parts_output_layouts(out_dtype, d, window):
    a = make(1, 4, 2, 150, d, 32, [5000], seed=79)
    a["window"] = window
    want, want_lse = call(a, out_dtype)
    check(a, want, want_lse)
    for buf, view in ((torch.full((1, 150, 4, d), 7.0, dtype=out_dtype, device=dev()), lambda t: t.transpose(1, 2)),
                      (torch.full((1, 4, 150, d + 3), 7.0, dtype=out_dtype, device=dev()), lambda t: t[..., 1:d + 1]),
                      (torch.full((1, 4, d, 150), 7.0, dtype=out_dtype, device=dev()), lambda t: t.transpose(2, 3))):
        out, lse = view(buf), torch.empty((1, 4, 150, 2), device=dev())[..., 1]
        blkattn.fwd_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["pos"], a["scale"], out, lse,
                          window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        if buf.shape[-1] == d + 3:
            assert bool((buf[..., 0] == 7).all()) and bool((buf[..., d + 1:] == 7).all())


@pytest.mark.parametrize("Hq,Hkv,Tq,d,dtype", [(4, 2, 100, 128, BF16), (4, 2, 100, 64, BF16), (8, 2, 3, 128, BF16),
                                               (8, 2, 3, 64, BF16), (8, 2, 3, 128, F32), (8, 2, 9, 64, F32)])
def test_a_row_of_nan_stays_its_own(Hq, Hkv, Tq, d, dtype):
    a = make(2, Hq, Hkv, Tq, d, 16, [3000, 900], dtype, seed=101)
    want, want_lse = call(a)
    a["q"][0, 1, 2] = math.nan
    out, lse = call(a)
    if dtype == BF16:  # (the fp32 kernels take a row without a comparable score for an empty one)
        assert bool(torch.isnan(out[0, 1, 2]).all())
    rest = torch.ones(out.shape[:3], dtype=torch.bool, device=out.device)
    rest[0, 1, 2] = False
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


def test_prompts_in_parts_in_a_graph():
    a = make(2, 4, 2, 200, 128, 16, [4000, 3000], seed=83)
    out, lse = torch.empty_like(a["q"]), torch.empty(a["q"].shape[:3], device=dev())

    def run():
        blkattn.fwd_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["pos"], a["scale"], out, lse)

    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
        run()  # (the second joins after the first: one workspace)
    for shift in (0, 900, 3900):
        out.fill_(9.0)
        lse.fill_(9.0)
        g.replay()
        check(a, out, lse)
        a["lens"] -= 900
        a["pos"] -= 900


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Tq,d,window", [(1, 128, 1), (1, 64, 100), (5, 128, 128), (3, 64, 1000), (65, 128, 1),
                                         (300, 128, 200), (129, 128, 5000), (100, 64, 37),
                                         (300, 64, 200), (260, 64, 1)])
def test_window(Tq, d, window, dtype):
    # rows before every window were given back: their pages hold NaN and their entries -1
    lens = [1500, max(Tq, 129), max(Tq, 4)]
    a = make(3, 4, 2, Tq, d, 16, lens, dtype, seed=window)
    a["window"] = window
    for b, n in enumerate(lens):
        first = max(0, n - Tq - window + 1)
        for t in range(first // 16 * 16, first):
            a["kp"][int(a["table"][b, t // 16]), :, t % 16] = math.nan
            a["vp"][int(a["table"][b, t // 16]), :, t % 16] = math.nan
        a["table"][b, :first // 16] = -1
    check(a, *call(a))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("Tq,lens", [(1, [1, 40]), (6, [6, 133]), (6, [300, 258]), (31, [128, 129]), (64, [64, 200])])
def test_tree(Tq, lens, dtype, d):
    g = torch.Generator().manual_seed(Tq)
    a = make(2, 8, 2, Tq, d, 16, lens, dtype, seed=50 + Tq)
    tree = torch.zeros(2, Tq, dtype=torch.int64)
    for b in range(2):
        for i in range(Tq):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            m = (int(tree[b, parent]) & (2 ** 64 - 1)) if parent >= 0 else 0
            m |= 1 << i
            tree[b, i] = m - 2 ** 64 if m >= 2 ** 63 else m
    absent = Tq // 3  # nodes that were never appended: NaN rows that no live row lists
    pos = (a["lens"][:, None] - 1).expand(2, Tq).clone()
    for i in range(Tq - absent, Tq):
        pos[1, i] = -1
        t = lens[1] - Tq + i
        for pool in (a["kp"], a["vp"]):
            pool[int(a["table"][1, t // 16]), :, t % 16] = math.nan
    a["tree"], a["pos"] = tree.to(dev()), pos.to(torch.int32)
    check(a, *call(a))


@pytest.mark.parametrize("dtype,Tq,d,P", [(BF16, 1, 128, 16), (BF16, 4, 64, 8), (BF16, 100, 128, 32), (F32, 2, 128, 64),
                                          (BF16, 3, 128, 128), (BF16, 200, 128, 256), (F32, 1, 64, 16),
                                          (BF16, 150, 64, 16)])
def test_entries_without_a_page(dtype, Tq, d, P):
    lens = [1300, 700, 3 * P + 1]
    a = make(3, 4, 2, Tq, d, P, lens, dtype, seed=9)
    N = a["kp"].shape[0]
    for b, bad in ((0, [0, 2]), (1, [1])):
        for i, e in enumerate(bad):
            a["table"][b, e] = (-1, N, 2 ** 31 - 1)[i % 3]
    a["table"][2, :] = -5  # no page at all: every row is empty
    a["pos"][0, 0] = -1
    check(a, *call(a))


def test_positions_at_the_edges():
    a = make(4, 8, 2, 4, 128, 16, [300, 300, 300, 300], seed=11)
    a["pos"] = torch.tensor([[-1, 0, 299, 2 ** 31 - 1], [5, 4, 3, 2], [-(2 ** 31), 1000, 128, 127],
                             [-1, -1, -1, -1]], dtype=torch.int32, device=dev())
    check(a, *call(a))
    a["lens"] = torch.tensor([0, -5, 2 ** 31 - 1, 17], dtype=torch.int32, device=dev())
    a["table"][2] = a["table"][1].clone()
    a["table"][2, 19:] = -1  # the length passes the table: clamped, and no page there
    a["kp"].nan_to_num_(0.5)
    a["vp"].nan_to_num_(0.5)
    check(a, *call(a))


@pytest.mark.parametrize("d,P,Tq", [(128, 8, 1), (128, 64, 5), (128, 256, 40)])
def test_same_bits_as_the_contiguous_cache(d, P, Tq):
    # one arithmetic on units that no CTA boundary splits (longer ones may be
    # cut elsewhere, and prompts sum the weights before rounding them)
    lens = [128, 77]
    a = make(2, 8, 2, Tq, d, P, lens, seed=13, poison=False)
    K = a["table"].shape[1] * P
    k, v = (torch.zeros(2, 2, K, d, dtype=BF16, device=dev()) for _ in range(2))
    for b, n in enumerate(lens):
        ids = a["table"][b, : -(-n // P)].long()
        k[b, :, :len(ids) * P] = a["kp"][ids].transpose(0, 1).reshape(2, -1, d)
        v[b, :, :len(ids) * P] = a["vp"][ids].transpose(0, 1).reshape(2, -1, d)
    out, lse = call(a)
    want, want_lse = blkattn.attention(a["q"], k, v, a["lens"], a["pos"])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("Tq,d,dtype", [(1, 128, BF16), (5, 64, BF16), (200, 128, BF16), (3, 64, F32)])
def test_same_bits_whatever_the_pages(Tq, d, dtype):
    a = make(2, 8, 2, Tq, d, 16, [900, 333], dtype, seed=14, poison=False)
    want = call(a)
    for P, rows_major in ((8, True), (64, False), (256, True)):
        n = -(-a["table"].shape[1] * 16 // P)
        rows = {}
        for name in ("kp", "vp"):
            x = a[name][a["table"].long().clamp(0, a[name].shape[0] - 1)]          # [B, entries, H, 16, d]
            x = x.permute(0, 1, 3, 2, 4).reshape(2, -1, 2, d)                        # [B, keys, H, d]
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * P - x.shape[1]))
            x = x.reshape(2 * n, P, 2, d).flip(0)                                    # pages in another order
            rows[name] = x.transpose(1, 2) if rows_major else x.transpose(1, 2).contiguous()
        table = torch.arange(2 * n - 1, -1, -1, dtype=torch.int32, device=dev()).reshape(2, n)
        out, lse = call(dict(a, table=table, **rows))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Tq,d,dtype", [(1, 128, BF16), (6, 128, BF16), (90, 128, BF16), (2, 64, BF16), (2, 128, F32)])
def test_same_bits_whatever_the_pool_layout(Tq, d, dtype):
    # packed heads, packed rows, gaps behind every row, page part or head, K and V laid out differently
    a = make(2, 8, 2, Tq, d, 16, [500, 333], dtype, seed=15)
    want = call(a)
    N = a["kp"].shape[0]

    def padded(t, rows=0, dims=0, heads=0):
        buf = torch.full((N, 2 + heads, 16 + rows, d + dims), math.nan, dtype=dtype, device=dev())
        buf[:, :2, :16, :d] = t
        return buf[:, :2, :16, :d]

    def by_rows(t, heads=0):
        buf = torch.full((N, 16, 2 + heads, d), math.nan, dtype=dtype, device=dev())
        buf[:, :, :2] = t.transpose(1, 2)
        return buf[:, :, :2].transpose(1, 2)

    k, v = a["kp"], a["vp"]
    for kp, vp in ((padded(k, rows=8), padded(v, rows=8)), (padded(k, dims=8), padded(v, dims=8)),
                   (padded(k, heads=1), padded(v, heads=1)), (by_rows(k), by_rows(v)),
                   (by_rows(k, 3), by_rows(v, 3)), (by_rows(k), padded(v)), (padded(k, dims=64, rows=3), by_rows(v))):
        out, lse = call(dict(a, kp=kp, vp=vp))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_strided_views_and_shared_pages():
    a = make(2, 8, 2, 3, 64, 16, [200, 200], seed=17)
    a["table"][1] = a["table"][0]  # the same pages under both sequences
    want = call(a)
    check(a, *want)
    wide = torch.zeros(2, 3, 8, 70, dtype=BF16, device=dev())  # query rows that are not 16-byte aligned
    b = dict(a, q=wide[..., 3:67].transpose(1, 2))
    b["q"].copy_(a["q"])
    check(b, *call(b))
    t2 = torch.zeros(a["table"].shape[1], 2, 3, dtype=torch.int32, device=dev())
    t2[:, :, 1] = a["table"].t()
    l2 = torch.zeros(2, 5, dtype=torch.int32, device=dev())
    l2[:, 2] = a["lens"]
    c = dict(a, table=t2[:, :, 1].t(), lens=l2[:, 2], pos=a["pos"].t().contiguous().t())
    out = torch.full((2, 3, 8, 130), 7.0, dtype=BF16, device=dev())
    lse = torch.full((2, 8, 3, 2), 7.0, device=dev())
    blkattn.fwd_paged(c["q"], c["kp"], c["vp"], c["table"], c["lens"], c["pos"], c["scale"],
                      out[..., 1:65].transpose(1, 2), lse[..., 0])
    check(c, out[..., 1:65].transpose(1, 2), lse[..., 0])
    assert bool((out[..., 0] == 7).all()) and bool((out[..., 65:] == 7).all()) and bool((lse[..., 1] == 7).all())
    both = torch.zeros(a["kp"].shape[0], 2, 2, 16, 64, dtype=BF16, device=dev())  # K and V of a page side by side
    both[:, 0], both[:, 1] = a["kp"], a["vp"]
    e = dict(a, kp=both[:, 0], vp=both[:, 1])
    got = call(e)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("Tq,d,dtype", [(1, 128, BF16), (70, 128, BF16), (2, 64, BF16), (1, 64, F32)])
def test_strides_of_single_dims_do_not_matter(Tq, d, dtype):
    # one sequence, one KV head, one page of 512 rows: every such dim with a stride of 0 or of no alignment
    a = make(1, 4, 1, Tq, d, 512, [300], dtype, seed=20, spare=0, entries=1)
    want = call(a, dtype)
    check(a, *want)

    def odd(t, s):
        return t.as_strided(t.shape, [x if n > 1 else s for n, x in zip(t.shape, t.stride())])

    for s in (0, 1, 7):
        b = dict(a, q=odd(a["q"], s), kp=odd(a["kp"], s), vp=odd(a["vp"], s), table=odd(a["table"], s),
                 pos=odd(a["pos"], s), lens=odd(a["lens"], s))
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        blkattn.fwd_paged(b["q"], b["kp"], b["vp"], b["table"], b["lens"], b["pos"], b["scale"], odd(out, s), odd(lse, s))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("d,window", [(128, 0), (64, 0), (128, 90), (64, 90)])
def test_prompt_output_layouts(out_dtype, d, window):
    a = make(1, 4, 2, 150, d, 32, [400], seed=19)
    a["window"] = window
    want, want_lse = call(a, out_dtype)
    check(a, want, want_lse)
    for buf, view in ((torch.full((1, 150, 4, d), 7.0, dtype=out_dtype, device=dev()), lambda t: t.transpose(1, 2)),
                      (torch.full((1, 4, 150, d + 3), 7.0, dtype=out_dtype, device=dev()), lambda t: t[..., 1:d + 1]),
                      (torch.full((1, 4, 150, d + 8), 7.0, dtype=out_dtype, device=dev()), lambda t: t[..., 8:])):
        out, lse = view(buf), torch.empty_like(want_lse)
        blkattn.fwd_paged(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["pos"], a["scale"], out, lse,
                          window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("window", [0, 40])
def test_more_sequences_than_the_unit_table(window):
    B = 1100
    a = make(B, 4, 2, 1, 64, 8, [1 + (7 * b) % 90 for b in range(B)], seed=23)
    a["window"] = window
    check(a, *call(a, BF16))


def test_wide_groups_and_large_scales():
    a = make(1, 128, 1, 2, 128, 16, [777], seed=29)
    check(a, *call(a))
    a = make(2, 8, 2, 1, 128, 16, [500, 900], seed=31, sharp=8.0)
    check(a, *call(a))
    for s in (-0.05, 0.0):
        a["scale"] = s
        check(a, *call(a))
    a = make(1, 4, 2, 70, 128, 16, [200], seed=37)
    for s in (-0.05, 0.0):  # a prompt that the prompt kernel does not take
        a["scale"] = s
        check(a, *call(a))


def test_long_context():
    a = make(1, 8, 2, 1, 128, 64, [70001], seed=41)
    check(a, *call(a, BF16))


@pytest.mark.parametrize("Tq,P,n", [(64, 65536, 129), (64, 32768, 70), (1, 32768, 70)])
def test_very_long_prompts_and_contexts(Tq, P, n):
    # one page, n times in the table (129 x 65536 keys are past the decode
    # kernel's range): the attention of one page's keys, lse + ln n
    a = make(1, 1, 1, Tq, 64, P, [P], seed=89)
    a["vp"] += 3  # outputs well away from 0
    ro, rl, ob, lb = reference(dict(a, pos=torch.full_like(a["pos"], P - 1)))
    a["table"] = a["table"][:, :1].repeat(1, n)
    a["lens"] = a["lens"] * n
    a["pos"] = torch.full_like(a["pos"], n * P - 1)
    out, lse = call(a)
    assert blkattn.check_device_error() == 0
    # One sequence is cut into 16 parts or more.  Within one, l takes a sum a
    # tile of 128 keys (2^-24 each), U a product of 16 keys (2^-23 each).
    more_l = n * P / 16 / 128 * 2.0 ** -24
    more_u = n * P / 16 / 16 * 2.0 ** -23
    av = float(a["vp"][int(a["table"][0, 0])].double().abs().max())
    assert bool(((out.double() - ro).abs() <= ob + (more_l + more_u) * av + 2.0 ** -24 * ro.abs()).all())
    assert bool(((lse.double() - rl - math.log(n)).abs() <= lb + more_l + 2.0 ** -21 * math.log(n)).all())


@pytest.mark.parametrize("Tq", [1, 100])
def test_pool_offsets_past_32_bits(Tq):
    P, H, d = 256, 8, 128
    N = (1 << 31) // (P * H * d) + 2
    kp = torch.zeros((N, P, H, d), dtype=BF16, device=dev()).transpose(1, 2)
    vp = torch.zeros((N, H, P, d), dtype=BF16, device=dev())
    small = make(1, 8, H, Tq, d, P, [600], seed=43, poison=False)
    ids = [N - 1, 3, N - 2]
    for i, pg in enumerate(ids):
        kp[pg], vp[pg] = small["kp"][int(small["table"][0, i])], small["vp"][int(small["table"][0, i])]
    ids += [-1] * (small["table"].shape[1] - len(ids))  # (the same T_max: the keys are cut alike)
    a = dict(small, kp=kp, vp=vp, table=torch.tensor([ids], dtype=torch.int32, device=dev()))
    out, lse = call(a)
    want, want_lse = call(small)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("Tq,d", [(1, 128), (5, 64), (80, 128)])
def test_graph_and_side_stream(Tq, d):
    a = make(2, 8, 2, Tq, d, 16, [300, 200], seed=47)
    check(a, *call(a))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call(a, BF16)
    b = make(2, 8, 2, Tq, d, 16, [300, 200], seed=48)
    for n in ("q", "kp", "vp", "table", "pos"):
        a[n].copy_(b[n])
    a["lens"] -= 1
    g.replay()
    torch.cuda.synchronize()
    check(a, out, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = call(a, BF16, stream=s)
    s.synchronize()
    check(a, out, lse)


# --------------------------------------------------------- used together
def test_serving_steps():
    """Prompt in chunks, then single tokens: append and attend over pages, as
    a serving loop runs them, equal to one pass over the whole sequence."""
    B, Hq, Hkv, d, P, T = 2, 8, 2, 128, 16, 150
    g = torch.Generator().manual_seed(60)
    q, k, v = (torch.randn(B, T, h, d, generator=g).to(BF16).transpose(1, 2).to(dev()) for h in (Hq, Hkv, Hkv))
    w, mscale = blkattn.rope_angles(d, scaling="ramp", factor=4.0, trained=64.0, low=1.0, high=4.0)
    ph = blkattn.rope_phases(w)
    pages = -(-T // P)
    order = torch.randperm(B * pages, generator=g).to(torch.int32).reshape(B, pages)
    table = torch.full((B, pages), -1, dtype=torch.int32, device=dev())
    kp, vp = (torch.full((B * pages, P, Hkv, d), math.nan, dtype=BF16, device=dev()).transpose(1, 2) for _ in range(2))
    outs, at = [], 0
    for n in (70, 40, 33, 1, 1, 5):  # the last 5: verified drafts
        end = at + n
        table[:, at // P:-(-end // P)] = order[:, at // P:-(-end // P)].to(dev())  # pages as they are needed
        pos = torch.arange(at, end, dtype=torch.int32, device=dev()).expand(B, n)
        qr = blkattn.paged_append(k[:, :, at:end], v[:, :, at:end], pos, table, kp, vp, phases=ph, mscale=mscale,
                                  q=q[:, :, at:end])
        lens = torch.full((B,), end, dtype=torch.int32, device=dev())
        outs.append(blkattn.attention_paged(qr, kp, vp, table, lens, pos))
        at = end
    assert at == T
    pos = torch.arange(T, dtype=torch.int32, device=dev()).expand(B, T)
    qr, kr = (blkattn.rope(x, pos, ph, mscale=mscale) for x in (q, k))
    a = dict(q=qr, kp=kr, vp=v.contiguous(), table=torch.arange(B, dtype=torch.int32, device=dev())[:, None],
             lens=torch.full((B,), T, dtype=torch.int32, device=dev()), pos=pos, scale=d ** -0.5, tree=None, window=0)
    # the whole sequence as one reference (a page of T rows), for every row of every step
    ro, rl, ob, lb = reference(a)
    out, lse = torch.cat([o for o, _ in outs], 2), torch.cat([s for _, s in outs], 2)
    assert bool(((out.double() - ro).abs() <= ob * (1 + 2.0 ** -8) + 2.0 ** -24 * ro.abs()).all())
    assert bool(((lse.double() - rl).abs() <= lb).all())


def test_training_step():
    """rope, attention, its backward, rope's backward: dq and dk of the
    unrotated rows against autograd in 64 bits.

    The attention's backward takes P and dS as bf16 (2^-8 each) and the
    rotated rows are bf16 too, as every operand; its own tests hold dq to
    2^-7 of sum |dS||k| + 1e-6 of its largest.  The rotation mixes two dims of
    a row: the bound is that of both dims' sum, plus the rotation's 6.2e-7."""
    B, H, T, d = 1, 2, 200, 128
    g = torch.Generator().manual_seed(61)
    q, k, v, do = (torch.randn(B, H, T, d, generator=g).to(BF16).to(dev()) for _ in range(4))
    ph = blkattn.rope_phases(blkattn.rope_angles(d)[0])
    pos = torch.arange(T, dtype=torch.int32, device=dev()).expand(B, T)
    lens = torch.full((B,), T, dtype=torch.int32, device=dev())
    qr, kr = blkattn.rope(q, pos, ph), blkattn.rope(k, pos, ph)
    out, lse = blkattn.attention(qr, kr, v, lens, pos)
    dqr, dkr, dv = blkattn.attention_backward(qr, kr, v, lens, pos, out, lse, do)
    dq, dk = blkattn.rope_backward(dqr, pos, ph), blkattn.rope_backward(dkr, pos, ph)
    # gradients of the rotated rows in 64 bits, turned back by autograd through a 64-bit rotation
    ang = (pos.cpu().long()[:, :, None] * blkattn.rope_phases(blkattn.rope_angles(d)[0], device="cpu")).double()
    ang = ang[:, None] * (2 * math.pi / 2.0 ** 64)
    c, s = torch.cos(ang), torch.sin(ang)

    def turn(x):
        u, w = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((u * c - w * s, u * s + w * c), -1)

    leaf = [torch.zeros(B, H, T, d, dtype=F64, requires_grad=True) for _ in range(2)]
    # the operands the kernels saw (bf16 after the rotation), with the rotation's own derivative
    Q, K = (x.double().cpu() + turn(z) for x, z in zip((qr, kr), leaf))
    S = (Q @ K.transpose(2, 3)) * d ** -0.5
    S = S.masked_fill(~torch.ones(T, T, dtype=torch.bool).tril(), -math.inf)
    Pm = torch.softmax(S, -1)
    O = Pm @ v.double().cpu()
    O.backward(do.double().cpu())
    dP = do.double().cpu() @ v.double().cpu().transpose(2, 3)
    dS = (Pm * (dP - (do.double().cpu() * O).sum(-1, keepdim=True))).detach().abs()
    aq = dS @ kr.double().cpu().abs() * d ** -0.5
    ak = dS.transpose(2, 3) @ qr.double().cpu().abs() * d ** -0.5
    for got, want, ab in ((dq, leaf[0].grad, aq), (dk, leaf[1].grad, ak)):
        pair = ab[..., :d // 2] + ab[..., d // 2:]
        tol = (2.0 ** -7 + 6.2e-7) * torch.cat((pair, pair), -1) + 2e-6 * float(ab.max())
        err = (got.double().cpu() - want).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
