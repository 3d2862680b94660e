"""Attention over the 8-bit cache at its edges: rows of the cache that no query
row sees, every width of the row groups, batches and prompts cut into slices,
other streams and threads, and random problems.  Bounds as in
test_gpu_paged_q8.py."""
import math
import random
import threading

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_paged_q8 import BF16, E8, F8, F32, I32, U8, call, chain, check, make
from test_gpu_rotary import dev

pytestmark = pytest.mark.gpu


def poison(a, seen):
    """A copy of the problem whose cache is NaN, numbers and scales, in every row (block of rows) of a sequence's
    pages that `seen` [B, keys] has not."""
    b = dict(a)
    P, S = a["kp"].shape[2], a["kp"].shape[2] // a["ks"].shape[2]
    for n in ("kp", "vp", "ks", "vs"):
        b[n] = a[n].view(U8).clone()
    for i in range(a["table"].shape[0]):
        for j in range(0, seen.shape[1], P):
            page = int(a["table"][i, j // P])
            rows = seen[i, j:j + P]
            rows = torch.nn.functional.pad(rows, (0, P - rows.numel()))
            hole = (~rows).nonzero()[:, 0].to(dev())
            blocks = (~rows.view(-1, S).any(1)).nonzero()[:, 0].to(dev())
            for n in ("kp", "vp"):
                b[n][page, :, hole] = 0x7f
            for n in ("ks", "vs"):
                b[n][page, :, blocks] = 255
    for n, t in (("kp", F8), ("vp", F8), ("ks", E8), ("vs", E8)):
        b[n] = b[n].view(t)
    return b


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("d,Hq,Tq,P,S", [(64, 4, 1, 16, 1), (128, 4, 1, 16, 1), (128, 8, 3, 32, 4), (128, 16, 2, 8, 8),
                                         (128, 8, 5, 16, 1), (128, 2, 70, 16, 2), (64, 2, 64, 32, 32)])
@pytest.mark.parametrize("mode", ["past", "window", "both"])
def test_unseen_rows_hold_anything(mode, d, Hq, Tq, P, S, out):
    n, end = 900, 900 if mode == "window" else 613
    a = make(2, Hq, 1, Tq, d, P, S, [n, n], spread=0, heads_first=Tq >= 64)
    a["pos"] = (end - Tq + torch.arange(Tq, device=dev(), dtype=I32)).expand(2, Tq).contiguous()
    a["window"] = 0 if mode == "past" else 77
    j = torch.arange(n)
    seen = ((j < end) & (j > (end - Tq - 77 if a["window"] else -1))).expand(2, n)
    want = call(a, out)
    check(a, want, out)
    for x, y in zip(call(poison(a, seen), out), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_unlisted_tree_nodes_hold_anything(d, out):
    n, T = 700, 6
    a = make(2, 8, 2, T, d, 16, 1, [n, n], spread=0)
    a["pos"][:] = n - 1
    a["tree"] = torch.tensor([1, 1, 9, 9, 41, 41], device=dev()).expand(2, T).contiguous()  # (nodes 0, 3 and 5)
    seen = torch.ones(2, n, dtype=torch.bool)
    for node in (1, 2, 4):
        seen[:, n - T + node] = False
    want = call(a, out)
    check(a, want, out)
    for x, y in zip(call(poison(a, seen), out), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("mode", ["causal", "window", "tree"])
@pytest.mark.parametrize("G,T", [(1, 1), (8, 1), (3, 3), (8, 2), (17, 1), (5, 5), (16, 2), (11, 3), (8, 5), (16, 3), (7, 7),
                                 (16, 4), (12, 8), (20, 5)])
def test_every_width_of_row_groups(G, T, mode):
    """Heads of 128 with a bf16 out over more than 256 keys: 1 to 100 rows a KV head."""
    a = make(3, 2 * G, 2, T, 128, 16, 8, [1 + T, 900, 2333], seed=G + T)
    if mode == "window":
        a["window"] = 200
    if mode == "tree":
        a["pos"][:] = a["lens"][:, None] - 1
        a["tree"] = torch.tensor(chain(T), device=dev()).expand(3, T).contiguous()
    a["pos"][1, 0] = -1
    check(a, call(a, BF16), BF16)


def test_scales_far_apart_in_many_rows():
    a = make(1, 40, 1, 1, 128, 16, 16, [1600], spread=12)
    check(a, call(a, BF16), BF16)
    a["vs"].view(U8)[int(a["table"][0, 3])] = 200
    check(a, call(a, BF16), BF16)
    a["vs"].view(U8)[int(a["table"][0, 3])] = 20
    a["ks"].view(U8)[int(a["table"][0, 70])] = 90
    check(a, call(a, BF16), BF16)


def test_rows_of_any_size_and_nan():
    a = make(1, 8, 1, 2, 128, 16, 16, [2000])
    size = torch.tensor([1, 1e-30, 1e-37, 0, 1e4, 300, 1e-5, 7], device=dev())
    a["q"] = (a["q"].float() * size[None, :, None, None]).to(BF16)
    for s in (a["scale"], 0.0, -0.3):
        a["scale"] = s
        check(a, call(a, BF16), BF16)
    clean = call(a, BF16)
    for bad in (math.nan, math.inf):
        b = dict(a, q=a["q"].clone(), scale=0.1)
        clean = call(dict(a, scale=0.1), BF16)
        b["q"][0, 3, 1, 7] = bad
        out, lse = call(b, BF16)
        assert bool(out[0, 3, 1].isnan().all()) and bool(lse[0, 3, 1].isnan())
        for x, y in zip((out, lse), clean):
            x[0, 3, 1] = y[0, 3, 1]
            assert torch.equal(x, y)
    # a NaN among the keys: the rows that see it (the second of each head)
    b = dict(a, scale=0.1, kp=a["kp"].view(U8).clone().view(F8))
    b["kp"].view(U8)[int(a["table"][0, 1999 // 16]), 0, 1999 % 16, 5] = 0xff
    out, lse = call(b, BF16)
    assert bool(out[0, :, 1].isnan().all()) and bool(lse[0, :, 1].isnan().all())
    assert torch.equal(out[0, :, 0], clean[0][0, :, 0]) and torch.equal(lse[0, :, 0], clean[1][0, :, 0])


@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("byte", [40, 80, 127, 200, 235])
def test_all_values_small_or_large(byte, Hq):
    """Scales of V of 2^-87 to 2^108 throughout: weights go relative to the row's own."""
    a = make(1, Hq, 1, 1, 128, 16, 16, [1600], spread=0)
    a["vs"].view(U8)[a["vs"].view(U8) < 255] = byte
    check(a, call(a, BF16), BF16)
    check(a, call(a, F32), F32)
    a["q"] = a["q"] * 20  # (scores that rise by hundreds)
    check(a, call(a, BF16), BF16)


def test_batches_cut_into_launches():
    lens = [(i * 53) % 300 for i in range(1300)]
    a = make(1300, 2, 1, 1, 128, 8, 8, lens, entries=40)
    check(a, call(a, BF16), BF16)


def test_prompts_cut_into_slices():
    """Tables so long that the bf16 copies of a batch's pages pass one slice."""
    a = make(3, 2, 8 // 4, 64, 128, 64, 16, [300, 64, 500], entries=1 << 15, heads_first=True)
    check(a, call(a, BF16), BF16)


def test_prompt_after_a_prompt_of_nan():
    """What an earlier call left in the library's copy of the pages is not read."""
    a = make(2, 2, 1, 64, 128, 16, 16, [333, 128], heads_first=True)
    b = make(2, 2, 1, 64, 128, 16, 16, [2048, 2048], seed=1, heads_first=True)
    b["kp"].view(U8)[:] = 0x7f
    b["vp"].view(U8)[:] = 0x7f
    for w in (0, 90):
        a["window"] = w
        want = call(a, BF16)
        call(b, BF16)
        for x, y in zip(call(a, BF16), want):
            assert torch.equal(x, y)
        check(a, want, BF16)


def test_calls_on_another_stream():
    """Outputs belong to the call's stream, which the current one lags behind."""
    g = torch.Generator().manual_seed(4)
    a = make(2, 8, 2, 3, 128, 16, 8, [400, 900])
    pos = torch.arange(40, dtype=I32, device=dev()).repeat(2, 1)
    pos[1, 30:] = -1
    x = {h: torch.randn(2, h, 40, 128, generator=g).to(BF16).to(dev()) for h in (2, 8)}
    w = (1 + 0.2 * torch.randn(128, generator=g)).to(BF16).to(dev())
    ph = blkattn.rope_phases(blkattn.rope_angles(128)[0])
    cache = a["kp"], a["vp"], a["ks"], a["vs"]
    calls = [lambda **kw: blkattn.qk_norm_rope(x[8], x[2], w, w, pos, ph, **kw),
             lambda **kw: blkattn.qk_norm_rope_backward(x[8], x[2], x[8], x[2], w, w, pos, ph, **kw),
             lambda **kw: (blkattn.paged_append_q8(x[2], x[2], pos, a["table"], *(t.view(U8).clone().view(t.dtype) for t in cache),
                                                   phases=ph, k_weight=w, q_weight=w, q=x[8], **kw),),
             lambda **kw: blkattn.paged_read_q8(pos, a["table"], *cache, **kw),
             lambda **kw: call(a, BF16, **kw), lambda **kw: call(a, F32, **kw)]
    s = torch.cuda.Stream()
    for f in calls:
        want = f()
        torch.cuda.synchronize()
        junk = [torch.full_like(t, 7.0) for t in want]  # (memory that the next allocations may take)
        del junk
        torch.cuda.synchronize()
        if f is calls[2]:  # (its pools are copied on the current stream first)
            got = f(stream=s)
            torch.cuda.synchronize()
        else:
            torch.cuda._sleep(100_000_000)
            got = f(stream=s)
            with torch.cuda.stream(s):
                early = [t.clone() for t in got]
            s.synchronize()
            for u, v in zip(early, want):
                assert torch.equal(u, v)
            torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_threads_on_one_stream():
    probs = [make(2, 8, 2, 2, 128, 16, 8, [700, 1500], seed=1), make(1, 4, 1, 64, 128, 16, 16, [900], seed=2, heads_first=True),
             make(3, 4, 2, 1, 64, 16, 8, [100, 900, 300], seed=3), make(1, 40, 1, 1, 128, 32, 16, [4000], seed=4)]
    want = [[t.clone() for t in call(a, BF16)] for a in probs]
    torch.cuda.synchronize()
    wrong = []

    def run(k):
        torch.cuda.set_device(0)
        for _ in range(50):
            for x, y in zip(call(probs[k], BF16), want[k]):
                if not torch.equal(x, y):
                    wrong.append(k)

    ts = [threading.Thread(target=run, args=(k,)) for k in range(len(probs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong


@pytest.mark.parametrize("seed", range(80))
def test_random(seed):
    r = random.Random(seed)
    d = r.choice([64, 128, 128])
    P = r.choice([8, 16, 32, 64, 128, 256])
    S = min(P, r.choice([1, 2, 4, 8, 16, 32, 64, 128]))
    Hkv = r.choice([1, 1, 2, 3])
    Hq = Hkv * r.choice([1, 2, 4, 7, 8])
    Tq = r.choice([1, 1, 2, 3, 5, 8, 17, 64, 90])
    B = r.choice([1, 2, 3, 5])
    most = r.choice([200, 600, 3000])
    lens = [r.randint(Tq, Tq + most) for _ in range(B)]
    a = make(B, Hq, Hkv, Tq, d, P, S, lens, seed=seed, rows_major=r.random() < 0.3, sharp=r.choice([0.3, 1.0, 3.0]),
             spread=r.choice([0, 2, 10]), heads_first=r.random() < 0.5)
    mode = r.choice(["causal", "window", "tree", "holes"])
    if mode == "window":
        a["window"] = r.choice([1, 15, 128, 1000])
    elif mode == "tree" and Tq <= 64:
        a["pos"][:] = a["lens"][:, None] - 1
        masks = []
        for i in range(Tq):
            up = r.randrange(-1, i)
            m = (masks[up] if up >= 0 else 0) | 1 << i
            masks.append(m)
        masks = [m - (1 << 64) if m >= 1 << 63 else m for m in masks]
        a["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev()).expand(B, Tq).contiguous()
    elif mode == "holes":
        for b in range(B):
            a["table"][b, r.randrange(a["table"].shape[1])] = -1
        a["pos"][0, r.randrange(Tq)] = -1
    out = r.choice([BF16, BF16, F32])
    check(a, call(a, out), out)
