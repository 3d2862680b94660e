"""What the rounding of the weights may do to a paged prompt.

On a key tile that every row of the query tile sees, the prompt kernel's
weights are rounded to bf16: p' = p (1 + D), |D| <= 2^-8.  The output divides
by the sum of the rounded weights, so it stays a convex combination of the
values:

    o' - o = sum p D (v - o) / sum p',    |o' - o| <= 2^-8 sum p |v - o| / (sum p (1 - 2^-8)),

which vanishes where one key holds all the weight and where all values are the
same.  lse takes the sum before the rounding.  Everything else is as in
test_gpu_paged.py: a score is off by E = 2^-23 (d + 4) scale sum |q||k|, a
weight by 2^-16 + 2^-21 besides, n keys are summed in fp32 (2^-23 a step), so
the quotient is off by 2 e sum p |v| / sum p with e = E + 2^-16 + 2^-21 + n 2^-23,
and lse by e without the 2^-16 of the split weights, plus 2^-21 |lse|.
"""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_paged import BF16, call, make

pytestmark = pytest.mark.gpu


def exact(a, rounded):
    """(out, lse, bounds) of one sequence whose keys all have pages, in 64 bits."""
    q, table = a["q"].double(), a["table"].long()
    _, Hq, Tq, d = q.shape
    P, n = a["kp"].shape[2], int(a["lens"][0])
    G = Hq // a["kp"].shape[1]
    k, v = (a[x][table[0, : -(-n // P)]].double().transpose(0, 1).reshape(-1, (-(-n // P)) * P, d)[:, :n]
            .repeat_interleave(G, 0)[None] for x in ("kp", "vp"))
    z = q @ k.transpose(2, 3) * a["scale"]
    j = torch.arange(n, device=q.device)
    pos = a["pos"][0].long()[:, None]
    see = j[None] <= pos
    if a["window"]:
        see = see & (j[None] > pos - a["window"])
    E = (q.abs() @ k.abs().transpose(2, 3) * abs(a["scale"]) * 2.0 ** -23 * (d + 4)).masked_fill(~see, 0.0).amax(-1)
    z = z.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None])
    o = p @ v
    e = E + 2.0 ** -21 + n * 2.0 ** -23
    ob = 2 * (e + 2.0 ** -16)[..., None] * (p @ v.abs()) + 2.0 ** -24 * o.abs()
    if rounded:  # sum p |v - o|, a dim at a time
        for x in range(d):
            spread = (p * (v[..., None, :, x] - o[..., x, None]).abs()).sum(-1)
            ob[..., x] += 2.0 ** -8 / (1 - 2.0 ** -8) * spread
    return o, lse, ob, e + 2.0 ** -21 * lse.abs()


def check(a, rounded=True):
    out, lse = call(a)
    assert blkattn.check_device_error() == 0
    o, s, ob, lb = exact(a, rounded)
    err = (out.double() - o).abs()
    assert bool((err <= ob).all()), float((err / ob).max())
    le = (lse.double() - s).abs()
    assert bool((le <= lb).all()), float((le / lb).max())


def write(a, name, rows):
    """rows [Hkv, n, d] into the pages of the (only) sequence."""
    P = a[name].shape[2]
    for j, pg in enumerate(a["table"][0, : -(-rows.shape[1] // P)].tolist()):
        r = rows[:, j * P:(j + 1) * P]
        a[name][pg, :, :r.shape[1]] = r.to(a[name].dtype).to(a[name].device)


# whole items, and items in parts (a table much longer than the sequence)
CUT = [(130, 700, None), (130, 700, 190), (300, 1000, None), (300, 1000, 300)]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [0, 600])
@pytest.mark.parametrize("Tq,n,entries", CUT)
def test_one_dominant_key_in_a_later_tile(Tq, n, entries, window, d):
    # scores of 0 for one key of every tile and -12 for the others, but one key
    # of a later tile at 3.2 to 5.4: below the 8 / log2(e) at which a row's
    # reference rises, so its weight is no power of two and holds over 9/10
    a = make(1, 4, 2, Tq, d, 16, [n], BF16, seed=3, entries=entries)
    a["window"] = window
    e = torch.zeros(d)
    e[::2] = 1.0
    level = torch.full((n,), -12.0)
    level[::128] = 0.0
    at = n - Tq - 130  # (seen by every row, in a tile that every row sees)
    level[at] = 5.4
    write(a, "kp", (level[:, None] * e).expand(2, n, d) * (2.0 / d / a["scale"]))
    gain = torch.linspace(0.6, 1.0, 4 * Tq).reshape(1, Tq, 4, 1)
    a["q"].copy_((gain * e).to(BF16).transpose(1, 2))
    check(a)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [0, 600])
@pytest.mark.parametrize("Tq,n,entries", CUT)
def test_equal_values_come_back(Tq, n, entries, window, d):
    a = make(1, 4, 2, Tq, d, 16, [n], BF16, seed=5, entries=entries, sharp=3.0)
    a["window"] = window
    write(a, "vp", torch.linspace(-3.0, 3.0, d).expand(2, n, d))
    check(a)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("sharp", [1.0, 4.0])
@pytest.mark.parametrize("Tq,n,entries", CUT)
def test_random_rows(Tq, n, entries, sharp, d):
    check(make(1, 4, 2, Tq, d, 16, [n], BF16, seed=9, entries=entries, sharp=sharp))


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq,Tq,n,sign", [(1, 64, 40000, 1.0), (4, 70, 900, -1.0)])
def test_prompt_rows_on_the_decode_kernel(Hq, Tq, n, sign, d):
    # few rows over a long context, and a negative scale, go to the decode
    # kernel, which splits every weight: nothing of the 2^-8
    a = make(1, Hq, 1, Tq, d, 32, [n], BF16, seed=15)
    a["scale"] *= sign
    check(a, rounded=False)
