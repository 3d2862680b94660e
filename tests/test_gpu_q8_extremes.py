"""The 8-bit cache at the ends of its exponents and over long tails.  Bounds as
in test_gpu_paged_q8.py where nothing else is said."""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_paged_q8 import BF16, E8, F32, F64, F8, I32, U8, call, check, make
from test_gpu_rotary import dev

pytestmark = pytest.mark.gpu


def paged(x, S, byte, P=16):
    """Rows x [B, Hkv, n, d] of e4m3's numbers as (pool, scales) in table order, n a multiple of P; `byte` the scale
    of each row (of each block: its first row's)."""
    B, H, n, d = x.shape
    pool = x.view(B, H, n // P, P, d).transpose(1, 2).reshape(B * n // P, H, P, d).to(F8).contiguous()
    scale = byte.view(B, H, n // P, P // S, S)[..., 0].transpose(1, 2).reshape(B * n // P, H, P // S)
    return pool, scale.to(U8).contiguous().view(E8)


def problem(k, v, kb, vb, q, S, scale, P=16):
    B, H, n, d = k.shape
    kp, ks = paged(k, S, kb, P)
    vp, vs = paged(v, S, vb, P)
    table = torch.arange(B * n // P, dtype=I32, device=k.device).view(B, n // P)
    T = q.shape[2]
    pos = (n - T + torch.arange(T, device=k.device, dtype=I32)).expand(B, T).contiguous()
    return dict(q=q.to(BF16), kp=kp, ks=ks, vp=vp, vs=vs, table=table,
                lens=torch.full((B,), n, dtype=I32, device=k.device), pos=pos, scale=scale, tree=None, window=0)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("G", [1, 12, 40])
@pytest.mark.parametrize("byte", [250, 253, 254])
def test_largest_scales_of_values(byte, G, out):
    """V's scales up to 2^127, and scores (base 2: scale is ln 2) that rise by 20 to 24 after a CTA's first tiles: both
    references of a row at the top of their range."""
    g = torch.Generator(device=dev()).manual_seed(G)
    B, H, n, d = 16, 8, 2560, 128
    k = torch.zeros(B, H, n, d, device=dev())
    for h in range(H):
        for tile, t in (((7, 24.0),), ((3, 22.0), (7, 24.0)), ((3, 20.0), (5, 22.0), (7, 24.0)), ((6, 23.5),))[h % 4]:
            k[:, h, 256 * tile + 100, 0] = min(t, 16)
            k[:, h, 256 * tile + 100, 1] = max(t - 16, 0)
    v = (torch.randn(B, H, n, d, generator=g, device=dev()) / 8).clamp(-0.5, 0.5)
    q = torch.zeros(B, H * G, 1, d, device=dev())
    q[..., :2] = 1
    a = problem(k, v, torch.full((B, H, n), 127, device=dev()), torch.full((B, H, n), byte, device=dev()), q, 16,
                math.log(2.0))
    check(a, call(a, out), out)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 12), (128, 4), (128, 40)])
def test_small_rows_beside_large_keys(d, G, out):
    """Query rows of 2^-110 to 2^-133 and keys whose scales make their scores ordinary numbers again."""
    for e in (-110, -114, -120, -126, -130, -133):
        a = make(2, G, 1, 1, d, 16, 16, [200, 700], spread=0, seed=-e)
        a["ks"].view(U8)[a["ks"].view(U8) < 255] = min(254, 127 - e - 7)
        a["q"] = (a["q"].float().sign() * 2.0 ** (e + 60) * 2.0 ** -60).to(BF16)
        assert bool((a["q"] != 0).any())
        check(a, call(a, out), out)


@pytest.mark.parametrize("G", [4, 12, 24, 40])
@pytest.mark.parametrize("n,far", [(1 << 13, 17), (1 << 17, 17), (1 << 20, 20), (1 << 20, 22)])
def test_one_strong_key_and_a_long_tail(n, far, G):
    """A key that outweighs each other one by 2^far and a bit, and a tail of equal ones that has a good part of the mass
    all the same, in units that lie in one or two CTAs (as many sequences as fill the machine twice, over the same
    pages).  A weight keeps 11 bits (off by 2^-11 of itself) or a step of 2^-27 of the row's largest (off by 2^-28 of
    that): out = n p v / (1 + n p) is off by at most 2^-11 + 2^-28 / p of itself, its bf16 by 2^-8, and the fp32 sums
    and powers by 2^-20 and n / 32 steps of 2^-24."""
    d, P = 128, 128
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    worst = 0.0
    for part in (1.125, 1.375, 1.625, 1.875):
        k = torch.zeros(1, 1, n, d, device=dev())
        k[:, :, 1:, 0] = -(far - far % 2)
        k[:, :, 1:, 1] = part - 2 - far % 2
        v = torch.zeros(1, 1, n, d, device=dev())
        v[:, :, 1:] = 1 + torch.arange(d, device=dev()).remainder(8) / 8
        q = torch.zeros(B, G, 1, d, device=dev())
        q[..., :2] = 1
        one = torch.full((1, 1, n), 127, device=dev())
        a = problem(k, v, one, one, q[:1], 16, math.log(2.0), P=P)
        a.update(q=q.to(BF16), **{x: a[x].expand(B, -1).contiguous() for x in ("table", "pos")}, lens=a["lens"].expand(B).contiguous())
        p = math.exp(math.log(2.0) * (part - 2 - far))
        want = (n - 1) * p / (1 + (n - 1) * p) * v[0, 0, 1].to(F64)
        got, lse = call(a, BF16)
        bound = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -28 / p + 2.0 ** -20 + n / 32 * 2.0 ** -24
        err = float(((got.to(F64) - want).abs() / want).max())
        worst = max(worst, err / bound)
        assert float((lse.to(F64) - math.log1p((n - 1) * p)).abs().max()) < 2.0 ** -20 + n / 32 * 2.0 ** -24
    assert worst <= 1, worst


@pytest.mark.parametrize("d", [64, 128])
def test_small_scales_read_as_bf16(d):
    """Scales below 2^-124: a number may lie between bf16's, and is rounded once."""
    a = make(2, 2, 2, 1, d, 16, 1, [300, 77], spread=0)
    for n in ("ks", "vs"):
        live = a[n].view(U8) < 255
        a[n].view(U8)[live] = torch.arange(int(live.sum()), device=dev()).remainder(8).to(U8)
    pos = torch.arange(300, device=dev(), dtype=I32).expand(2, 300).contiguous()
    pos[1, 77:] = -1
    cache = a["kp"], a["vp"], a["ks"], a["vs"]
    exact = blkattn.paged_read_q8(pos, a["table"], *cache, out_dtype=F32)
    near = blkattn.paged_read_q8(pos, a["table"], *cache, out_dtype=BF16)
    for x, y in zip(exact, near):
        assert torch.equal(x.to(BF16), y) and bool((x != x.to(BF16).float()).any())


def test_append_to_very_many_heads():
    """As many KV heads as there may be, in blocks of 128 rows, and the query rows of a decode step with them."""
    H, d, P = 32767, 128, 128
    g = torch.Generator(device=dev()).manual_seed(1)
    kp, vp = (torch.zeros(1, H, P, d, dtype=U8, device=dev()).view(F8) for _ in range(2))
    ks, vs = (torch.full((1, H, 1), 255, dtype=U8, device=dev()).view(E8) for _ in range(2))
    k, v = (torch.randn(1, H, 2, d, generator=g, device=dev()).to(BF16) for _ in range(2))
    q = torch.randn(1, 70, 2, d, generator=g, device=dev()).to(BF16)
    w = (1 + 0.2 * torch.randn(d, generator=g, device=dev())).to(BF16)
    pos = torch.tensor([[0, 1]], dtype=I32, device=dev())
    table = torch.zeros(1, 1, dtype=I32, device=dev())
    ph = blkattn.rope_phases(blkattn.rope_angles(d)[0])
    got = blkattn.paged_append_q8(k, v, pos, table, kp, vp, ks, vs, phases=ph, q_weight=w, q=q)
    # the same rows, some heads at a time
    for h0 in range(0, H, 8000):
        h1 = min(H, h0 + 8000)
        kq, vq = (torch.zeros(1, h1 - h0, P, d, dtype=U8, device=dev()).view(F8) for _ in range(2))
        kc, vc = (torch.full((1, h1 - h0, 1), 255, dtype=U8, device=dev()).view(E8) for _ in range(2))
        want = blkattn.paged_append_q8(k[:, h0:h1], v[:, h0:h1], pos, table, kq, vq, kc, vc, phases=ph, q_weight=w, q=q)
        for x, y in ((kp, kq), (vp, vq), (ks, kc), (vs, vc)):
            assert torch.equal(x.view(U8)[:, h0:h1], y.view(U8))
    # (a decode step's query rows and a prompt's may differ in an fp32 angle's last bits)
    err = (got.float() - want.float()).abs()
    assert bool((err <= 2.0 ** -7 * want.float().abs() + 2.0 ** -16).all())
