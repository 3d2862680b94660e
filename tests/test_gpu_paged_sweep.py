"""Random calls of the paged attention against the explicit 64-bit softmax:
types, head dims, groups, page sizes and layouts, tables much wider than the
sequences, lengths from 0, padding rows, windows, trees, entries without a
page, broadcast and strided arguments."""
import math
import random

import pytest
import torch

from test_gpu_paged import BF16, F32, call, check, dev, make

pytestmark = pytest.mark.gpu


def log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(seed):
    rng = random.Random(seed)
    dtype = rng.choice((BF16, BF16, F32))
    d = rng.choice((64, 128))
    Hkv, G = rng.choice((1, 2, 3, 5, 8)), rng.choice((1, 2, 4, 7, 8))
    Tq = rng.choice((1, 1, 2, 3, 6, 9, 17, 33, 63, 64, 65, 100, 129, 257, 300))
    if Tq > 33:
        Hkv, G = min(Hkv, 3), min(G, 4)
    B = rng.randint(1, 2 if Tq > 60 else 5)
    P = rng.choice((8, 16, 16, 32, 64, 128, 256, 1024))
    lens = [rng.choice((0, Tq, Tq + rng.randint(0, 40), log(rng, 1, 4000), log(rng, 100, 4000))) for _ in range(B)]
    need = max(1, max(-(-n // P) for n in lens)) + 1
    entries = rng.choice((None, None, need + log(rng, 1, max(2, 40000 // P))))
    a = make(B, Hkv * G, Hkv, Tq, d, P, lens, dtype, rng.random() < 0.5, seed=seed, entries=entries,
             sharp=rng.choice((1.0, 1.0, 3.0)))
    kind = rng.choice(("plain", "plain", "window", "tree"))
    if kind == "window":
        a["window"] = log(rng, 1, 5000)
    if kind == "tree" and Tq <= 64:
        bits = [[rng.getrandbits(Tq) | 1 << i for i in range(Tq)] for _ in range(B)]
        a["tree"] = torch.tensor([[m - 2 ** 64 if m >= 2 ** 63 else m for m in row] for row in bits],
                                 dtype=torch.int64, device=dev())
        if rng.random() < 0.5:
            a["pos"] = torch.clamp(a["lens"][:, None] - 1, min=-1).expand(B, Tq)
    if rng.random() < 0.3:  # pages that are not there
        for b in range(B):
            for i in range(-(-lens[b] // P)):
                if rng.random() < 0.2:
                    a["table"][b, i] = rng.choice((-1, -2 ** 31, 2 ** 31 - 1, a["kp"].shape[0]))
    if rng.random() < 0.3:  # rows in another order, padding, positions past the end
        pos = a["pos"].clone()
        pos = pos[:, torch.randperm(Tq, generator=torch.Generator().manual_seed(seed)).to(dev())]
        for b in range(B):
            for i in range(Tq):
                x = rng.random()
                if x < 0.1:
                    pos[b, i] = rng.choice((-1, -2 ** 31))
                elif x < 0.2:
                    pos[b, i] += rng.choice((1, 50))
        a["pos"] = pos.contiguous()
    if rng.random() < 0.15:  # broadcast arguments
        a["q"] = a["q"][:, :1].expand(a["q"].shape)
    if rng.random() < 0.15:
        a["q"] = a["q"][:, :, :1].expand(a["q"].shape)
    if rng.random() < 0.15:
        a["q"] = a["q"].contiguous().transpose(2, 3).contiguous().transpose(2, 3)  # dims apart
    if rng.random() < 0.1:
        a["scale"] *= rng.choice((-1.0, 0.0, 4.0))
    return a, rng.choice((F32, BF16))


@pytest.mark.parametrize("seed", range(240))
def test_random_calls(seed):
    a, out_dtype = draw(seed)
    # (rows at random positions leave unseen keys between seen ones, whose rows
    # have to be finite)
    a["kp"].nan_to_num_(0.25)
    a["vp"].nan_to_num_(0.25)
    check(a, *call(a, out_dtype))


# one case for each kernel: finished, folded and joined decode units, rows of
# prompts whole and in parts, fp32 rows up to 8 a KV head and above
@pytest.mark.parametrize("B,Hq,Hkv,Tq,d,K,dtype", [
    (2, 4, 1, 1, 128, 90, BF16), (4, 32, 8, 1, 128, 2500, BF16), (1, 8, 2, 3, 64, 3000, BF16),
    (2, 48, 48, 130, 128, 600, BF16), (1, 4, 2, 100, 64, 3000, BF16), (2, 4, 2, 2, 128, 1500, F32),
    (1, 8, 2, 9, 64, 2000, F32)])
def test_two_captured_calls_share_the_workspace(B, Hq, Hkv, Tq, d, K, dtype):
    two = [make(B, Hq, Hkv, Tq, d, 16, [K - 7 * b for b in range(B)], dtype, seed=s, entries=300) for s in (1, 2)]
    want = [call(a) for a in two]
    graphs, outs = [], []
    for a in two:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(a))
        graphs.append(g)
    for turn in range(3):
        for g, got, w in zip(graphs, outs, want):
            for t in got:
                t.fill_(7.0)
            g.replay()
        for got, w in zip(outs, want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    two[0]["lens"] -= 40  # other values in the captured buffers
    two[0]["pos"] -= 40
    graphs[0].replay()
    check(two[0], *outs[0])
