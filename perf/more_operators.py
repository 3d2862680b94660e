"""Measured cases of the head norms with rotation and of the 8-bit paged cache.

Five operators: `norm` (RMS norm of each query and key head with the rotary
position in the same pass), `norm_bwd` (its gradient), `append` (new K/V rows
normed, rotated and quantised into an 8-bit paged cache, and the blocks that
changed read back), `read` (rows of the 8-bit cache as numbers) and `attend`
(attention over the 8-bit cache).  `run` computes each in its plain form
(elementary torch operations) or, with `own`, through the library's binding.
Shapes are the library's: rows [B, heads, T, d], pools [pages, KV heads, page
rows, d], page tables int32 [B, entries].

An 8-bit pool holds e4m3 numbers and one power of two (e8m0: the byte e + 127)
for each block of S rows of a page and head; a number stands for e4m3 2^e.  A
block's exponent is the least with all its numbers within 448 2^e; a call that
writes a block's first row begins the block anew, others keep or raise the
exponent, and rows already there are rounded again when it rises.
"""
import math
from fractions import Fraction

import torch

own = False

_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8, _E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_EPS = 1e-6


# ------------------------------------------------------------------- cases
def _norm(name, B, Hq, Hkv, T, d, rot, layout="half", dtype="bf16", out="bf16", bwd=False, first=0, scaled=False,
          token_major=True):
    return {"name": name, "op": "norm_bwd" if bwd else "norm", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d,
            "rot": rot, "layout": layout, "dtype": dtype, "out": out, "first": first, "scaled": scaled,
            "token_major": token_major}


def _append(name, B, Hq, Hkv, T, d, rot, page, S, lo, hi, layout="half", dtype="bf16", rows_major=False, ragged=False,
            norm=True):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "rot": rot, "page": page,
            "S": S, "lo": lo, "hi": hi, "layout": layout, "dtype": dtype, "rows_major": rows_major, "ragged": ragged,
            "norm": norm}


def _read(name, B, Hkv, d, page, S, lo, hi, out="bf16", rows_major=False):
    return {"name": name, "op": "read", "B": B, "Hkv": Hkv, "T": hi, "d": d, "page": page, "S": S, "lo": lo, "hi": hi,
            "out": out, "rows_major": rows_major}


def _attend(name, B, Hq, Hkv, T, d, page, S, lo, hi, kind="causal", window=0, rows_major=False, absent=0, out="bf16"):
    return {"name": name, "op": "attend", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "page": page, "S": S,
            "lo": lo, "hi": hi, "kind": kind, "window": window, "rows_major": rows_major, "absent": absent, "out": out}


def listed():
    return [
        # the query and key rows of one decode step of 32 sequences: the smallest call, latency counts
        _norm("norm_decode_step", 32, 32, 8, 1, 128, 128, first=8000),
        # the query and key rows of whole prompts, as a projection lays them out (token-major)
        _norm("norm_prompt", 2, 32, 8, 8192, 128, 128),
        # the backward pass of a training step: f32 gradients as the attention's backward writes them
        _norm("norm_bwd_prompt", 2, 32, 8, 8192, 128, 128, dtype="bf16", out="bf16", bwd=True),
        # odd sizes, part of the head, interleaved pairs, far scaled positions, 32-bit rows and gradients
        _norm("norm_bwd_far_part", 3, 6, 3, 1777, 64, 24, layout="interleaved", dtype="f32", out="f32", bwd=True,
              first=1000000, scaled=True, token_major=False),
        # one decode step of 32 sequences into small pages, a scale a page, with its query rows
        _append("append_decode_step", 32, 32, 8, 1, 128, 128, 16, 16, 512, 8191),
        # a chunk of prompts of different lengths (short ones padded), pages of 64 with two scales each
        _append("append_prompt_chunk", 4, 64, 8, 2048, 128, 128, 64, 32, 0, 2048, ragged=True),
        # the whole cache of one long context read back
        _read("read_long_p128", 1, 8, 128, 128, 128, 131072, 131072),
        # short prefixes of different lengths, heads of 64, token-wise scales, exact 32-bit numbers
        _read("read_prefixes_d64", 8, 4, 64, 16, 1, 100, 1777, out="f32", rows_major=True),
        # batched decode over small pages
        _attend("decode_batch_p16", 32, 32, 8, 1, 128, 16, 16, 512, 8192),
        # one long context, one page a tile, a scale for every 8 rows
        _attend("decode_long_p128", 1, 32, 8, 1, 128, 128, 8, 131072, 131072, rows_major=True),
        # verification of five-row chains, some rows absent
        _attend("verify_chain_p32", 8, 64, 8, 5, 128, 32, 32, 1024, 32768, absent=2),
        # the last 2048 rows of prompts, over the pages that hold all of them
        _attend("prompt_chunk_p64", 2, 32, 8, 2048, 128, 64, 64, 8192, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "append", "append", "read", "attend", "attend", "attend"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 7, 8))
    if op in ("norm", "norm_bwd"):
        T = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 64), (1 << 19) // (T * (G + 1) * Hkv)))
        case = _norm("", B, G * Hkv, Hkv, T, d, rng.choice((d, d, d // 2, 2 * rng.randint(1, d // 2))),
                     layout=rng.choice(("half", "interleaved")), dtype=rng.choice(("bf16", "bf16", "f32")),
                     out=rng.choice(("bf16", "f32")), bwd=op == "norm_bwd", first=_log(rng, 1, 1 << 21),
                     scaled=rng.random() < 0.5, token_major=rng.random() < 0.5)
        return {k: v for k, v in case.items() if k != "name"}
    page = rng.choice((8, 16, 16, 32, 64, 128, 256))
    S = 1 << rng.randint(0, min(7, page.bit_length() - 1))
    rows_major = rng.random() < 0.5
    if op == "append":
        T = _log(rng, 1, 2048)
        B = max(1, min(_log(rng, 1, 64), 2048 // T))
        lo = _log(rng, 1, 4096)
        case = _append("", B, G * Hkv, Hkv, T, d, rng.choice((0, d, d, d // 2)), page, S, lo,
                       lo + rng.randint(0, 2048), layout=rng.choice(("half", "interleaved")),
                       dtype=rng.choice(("bf16", "bf16", "f32")), rows_major=rows_major, ragged=rng.random() < 0.5,
                       norm=rng.random() < 0.5)
        return {k: v for k, v in case.items() if k != "name"}
    if op == "read":
        B = _log(rng, 1, 32)
        hi = _log(rng, 16, 131072 // B)
        case = _read("", B, Hkv, d, page, S, rng.randint(hi // 8, hi), hi, out=rng.choice(("bf16", "bf16", "f32")),
                     rows_major=rows_major)
        return {k: v for k, v in case.items() if k != "name"}
    kind = rng.choice(("causal", "causal", "tree", "window"))
    out = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind != "tree" and rng.random() < 0.3:
        out = "bf16"  # (what a prompt's next projection takes)
        T, B = _log(rng, 64, 2048), 1 if G * Hkv > 32 else rng.randint(1, 2)  # a prompt's chunk
        hi = _log(rng, T, 8192)
        lo = rng.randint(T, hi)
    else:
        T, B = rng.choice((1, 1, 2, 5, 8, 17)), _log(rng, 1, 32)
        hi = _log(rng, max(T, 16), 131072 // B)
        lo = rng.randint(max(T, hi // 8), hi)
    case = _attend("", B, G * Hkv, Hkv, T, d, page, S, lo, hi, kind="tree" if kind == "tree" else "causal",
                   window=_log(rng, 1, hi) if kind == "window" else 0, rows_major=rows_major,
                   absent=rng.randint(0, max(0, min(T - 1, 3))), out=out)
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------- numbers of a case
def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the same for every seed, in an order of its own for each."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tree_parents(T):
    """A small fixed tree: node i hangs below node (i - 1) // 2."""
    masks = []
    for i in range(T):
        m, n = 0, i
        while True:
            m |= 1 << n
            if n == 0:
                break
            n = (n - 1) // 2
        masks.append(m)
    return masks


def _angles(case):
    """w_i, the angle of one position for each pair, and the factor on both rotated parts.  Scaled: the slow
    pairs' angles divided by 8, the fast ones' kept, a linear ramp between (over the turns that each pair makes in
    the 8192 positions of the unscaled table)."""
    r = case["rot"]
    if r == 0:
        return [], 1.0
    w = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    if not case.get("scaled"):
        return w, 1.0
    out = []
    for x in w:
        turns = 8192 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        out.append(x * keep + x / 8.0 * (1.0 - keep))
    return out, 0.1 * math.log(8.0) + 1.0


def _phases(w):
    f = [int(Fraction(x) * (1 << 64) / _TWO_PI + Fraction(1, 2)) % (1 << 64) for x in w]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in f], dtype=torch.int64, device="cuda")


def _normal(g, shape, dtype):
    x = torch.empty(shape, dtype=torch.float32, device="cuda")
    return x.normal_(generator=g).to(dtype)


def _order(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _tables(g, lens, entries, page, spare):
    """Page tables whose pages lie in random order in a pool with a few spare pages (the last page is one); entries
    past a sequence's pages are -1."""
    need = [-(-n // page) for n in lens]
    N = sum(need) + spare
    order = _order(g, N - 1).to(torch.int32)
    table = torch.full((len(lens), max(1, entries)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, N


def _pool(g, N, Hkv, page, d, S, rows_major):
    """(numbers e4m3 [N, Hkv, page, d], scales e8m0 [N, Hkv, page / S]): normal values, each page and head with a size
    of its own, quantised as an append writes them."""
    size = torch.randint(-2, 3, (N, Hkv, 1, 1), generator=g, device="cuda")
    x = torch.empty((N, Hkv, page, d), dtype=torch.float32, device="cuda").normal_(generator=g)
    x = torch.ldexp(x, size).view(N, Hkv, page // S, S * d)
    m, ex = torch.frexp(x.abs().amax(3))
    e = ex - 9 + (m > 0.875)
    x = torch.ldexp(x, -e[..., None]).to(_F8).view(N, Hkv, page, d)
    if rows_major:
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    return x, (e + 127).to(torch.uint8).view(_E8)


def _rows(g, B, H, T, d, dtype, token_major=True):
    """[B, H, T, d], stored token by token as a projection writes them."""
    return _normal(g, (B, T, H, d), dtype).transpose(1, 2) if token_major else _normal(g, (B, H, T, d), dtype)


def _weights(g, d):
    """A norm's weight: near 1, as a trained one."""
    return (1.0 + 0.25 * _normal(g, (d,), torch.float32)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    B, T, d = case["B"], case["T"], case["d"]
    t = torch.arange(T, device="cuda")
    if case["op"] in ("norm", "norm_bwd"):
        dtype = _DT[case["dtype"]]
        w, s["mscale"] = _angles(case)
        s["w"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        s["phases"] = _phases(w)
        s["q"], s["k"] = (_rows(g, B, h, T, d, dtype) for h in (case["Hq"], case["Hkv"]))
        s["wq"], s["wk"] = _weights(g, d), _weights(g, d)
        start = torch.randint(0, case["first"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + t).to(torch.int32)
        if case["op"] == "norm_bwd":
            s["gq"], s["gk"] = (_rows(g, B, h, T, d, torch.float32, False) for h in (case["Hq"], case["Hkv"]))
        return s
    Hkv, page, S = case["Hkv"], case["page"], case["S"]
    lens = [_spread(case["lo"], case["hi"], B)[i] for i in _order(g, B).tolist()]
    if case["op"] == "append":
        dtype = _DT[case["dtype"]]
        w, s["mscale"] = _angles(case)
        s["w"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        s["phases"] = _phases(w) if w else None
        new = [_spread(max(1, T // 4), T, B)[i] for i in _order(g, B).tolist()] if case["ragged"] else [T] * B
        s["table"], N = _tables(g, [n + T for n in lens], -(-(case["hi"] + T + 2 * S) // page) + 1, page, 3)
        s["k_pages"], s["k_scales"] = _pool(g, N, Hkv, page, d, S, case["rows_major"])
        s["v_pages"], s["v_scales"] = _pool(g, N, Hkv, page, d, S, case["rows_major"])
        s["k"], s["v"], s["q"] = (_rows(g, B, h, T, d, dtype) for h in (Hkv, Hkv, case["Hq"]))
        s["wq"], s["wk"] = (_weights(g, d), _weights(g, d)) if case["norm"] else (None, None)
        s["q_out"] = torch.zeros((B, case["Hq"], T, d), dtype=dtype, device="cuda")
        first, n = (torch.tensor(v, device="cuda")[:, None] for v in (lens, new))
        s["pos"] = torch.where(t < n, first + t, -1).to(torch.int32)  # -1: a row that is padding
        # what is read back: the rows of the blocks that change, up to the last new one
        base = first // S * S
        i = torch.arange(T + S - 1, device="cuda")
        s["look"] = torch.where(base + i < first + n, base + i, -1).to(torch.int32)
        return s
    s["table"], N = _tables(g, lens, -(-case["hi"] // page), page, 3)
    s["k_pages"], s["k_scales"] = _pool(g, N, Hkv, page, d, S, case["rows_major"])
    s["v_pages"], s["v_scales"] = _pool(g, N, Hkv, page, d, S, case["rows_major"])
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "read":
        s["look"] = torch.where(t < s["lens"][:, None], t, -1).to(torch.int32)
        return s
    s["q"] = _rows(g, B, case["Hq"], T, d, torch.bfloat16)
    if case["kind"] == "tree":
        pos = (s["lens"][:, None] - 1).expand(B, T).clone()
        s["tree"] = torch.tensor(_tree_parents(T), dtype=torch.int64, device="cuda").expand(B, T).contiguous()
    else:
        pos = s["lens"][:, None] - T + t
        s["tree"] = None
    if case["absent"]:
        pos[B - 1, T - case["absent"]:] = -1  # the last sequence has fewer rows
    s["pos"] = pos.to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------ plain forms
def _cos_sin(s, sign=1):
    """cos and sin [B, 1, T, rot / 2] of the rows' angles, taken in 64 bits (32 lose those of far positions)."""
    a = sign * s["pos"].double()[:, None, :, None] * s["w"]
    return (torch.cos(a) * s["mscale"]).float(), (torch.sin(a) * s["mscale"]).float()


def _rotate(s, x, sign=1):
    rot = s["case"]["rot"]
    if rot == 0:
        return x
    cos, sin = _cos_sin(s, sign)
    y = x.clone()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if s["case"]["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., lo], x[..., hi]
    y[..., lo] = u * cos - v * sin
    y[..., hi] = u * sin + v * cos
    return y


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()


def _norm_gradient(s, g, x, w, dtype):
    """(dx, dw) of rows x normed with w and rotated, from the gradient g of the result."""
    g, x, w = _rotate(s, g.float(), -1), x.float(), w.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    h = x * r
    c = g * w
    dx = r * (c - h * (c * h).mean(-1, keepdim=True))
    return dx.to(dtype), (g * h).sum((0, 1, 2), dtype=torch.float64).float()


def _powers(e8):
    e = e8.view(torch.uint8).int() - 127
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _look(s, pages, scales, dtype):
    """The rows `look` of each sequence as numbers [B, Hkv, T, d]; zeros where it is negative."""
    c = s["case"]
    p = s["look"].long()
    page = s["table"].gather(1, (p.clamp(min=0) // c["page"])).long()
    row = p.clamp(min=0) % c["page"]
    x = pages.view(torch.uint8)[page, :, row].view(_F8).float()  # [B, T, Hkv, d]
    x = x * _powers(scales.view(torch.uint8)[page, :, row // c["S"]])[..., None]
    return torch.where((p >= 0)[:, :, None, None], x, 0.0).transpose(1, 2).to(dtype)


def _written(s, x, pages, scales):
    """Rows x [B, Hkv, T, d] in 32 bits quantised into the blocks that hold the rows `pos`."""
    c = s["case"]
    B, H, T, d = x.shape
    P, S = c["page"], c["S"]
    first, n = s["pos"][:, :1].long(), (s["pos"] >= 0).sum(1, keepdim=True)
    nb = -(-T // S) + 1  # blocks that T rows in a row can touch
    at = first // S * S + torch.arange(nb * S, device="cuda")
    ent = s["table"].gather(1, at // P).long()
    page, row = torch.where(ent < 0, pages.shape[0] - 1, ent), at % P  # (the spare page takes what no row needs)
    new = (at >= first) & (at < first + n)
    t = (at - first).clamp(0, T - 1)
    y = x.transpose(1, 2).gather(1, t[:, :, None, None].expand(-1, -1, H, d))  # [B, nb S, Hkv, d]
    y = torch.where(new[:, :, None, None], y, 0.0).view(B, nb, S, H, d)
    new = new.view(B, nb, S)
    size, byte = torch.where(torch.isfinite(y), y.abs(), 0.0).amax((2, 4)), pages.view(torch.uint8)
    m, ex = torch.frexp(size)
    e = torch.where(size == 0, -127, (ex - 9 + (m > 0.875)).clamp(min=-127))
    old = byte[page, :, row].view(B, nb, S, H, d)
    page0, block = page.view(B, nb, S)[:, :, 0], row.view(B, nb, S)[:, :, 0] // S
    e_old = scales.view(torch.uint8)[page0, :, block].int() - 127
    fresh = new[:, :, 0, None]
    e = torch.where(fresh, e, torch.maximum(e, e_old))
    kept = torch.ldexp(old.view(_F8).float(), (e_old - e)[:, :, None, :, None]).to(_F8).view(torch.uint8)
    kept = torch.where(fresh[:, :, None, :, None], old, kept)
    y = torch.ldexp(torch.where(torch.isfinite(y), y, math.nan), -e[:, :, None, :, None]).to(_F8).view(torch.uint8)
    touched = new.any(2)
    y = torch.where(new[..., None, None], y, torch.where(touched[:, :, None, None, None], kept, old))
    byte[page, :, row] = y.view(B, nb * S, H, d)
    scales.view(torch.uint8)[page0, :, block] = (torch.where(touched[:, :, None], e, e_old) + 127).to(torch.uint8)


def _gathered(pages, scales, table, S, T):
    """The cache rows of each sequence in order: [B, Hkv, T, d] in 32 bits (absent pages: page 0's rows, masked by the caller)."""
    B, n = table.shape
    ids = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[ids].view(_F8).float()  # [B, n, Hkv, page, d]
    H, page, d = x.shape[2:]
    x = x.reshape(B, n, H, page // S, S, d) * _powers(scales.view(torch.uint8)[ids])[..., None, None]
    return x.transpose(1, 2).reshape(B, H, n * page, d)[:, :, :T]


def _plain_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, d, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "page"))
    K = min(c["hi"], s["table"].shape[1] * page)
    k, v = (_gathered(s[n + "_pages"], s[n + "_scales"], s["table"], c["S"], K) for n in "kv")
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv * T, d)
    j = torch.arange(K, device="cuda")
    pos, lens = s["pos"].long()[:, :, None], s["lens"].long()[:, None, None]
    see = (j < lens) & (j <= pos)
    if c["window"]:
        see &= j > pos - c["window"]
    if s["tree"] is not None:
        node = j - (lens - T)
        see &= (node < 0) | ((s["tree"][:, :, None] >> node.clamp(0, 63)) & 1).bool()
    see = see[:, None].expand(B, Hq // Hkv, T, K).reshape(B, 1, Hq // Hkv * T, K)
    z = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    z = z.masked_fill_(~see, -math.inf)
    m = z.amax(dim=3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp_(z.sub_(m))
    l = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l)).reshape(B, Hq, T)
    return o.reshape(B, Hq, T, d).to(_DT[c["out"]]), lse


def run(s):
    c = s["case"]
    if own:
        from exact_blocked_attention_gb300 import blkattn
        if c["op"] == "norm":
            return blkattn.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["phases"], eps=_EPS,
                                        layout=c["layout"], mscale=s["mscale"], out_dtype=_DT[c["out"]])
        if c["op"] == "norm_bwd":
            return blkattn.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"],
                                                 s["phases"], eps=_EPS, layout=c["layout"], mscale=s["mscale"],
                                                 out_dtype=_DT[c["out"]])
        if c["op"] == "append":
            blkattn.paged_append_q8(s["k"], s["v"], s["pos"], s["table"], s["k_pages"], s["v_pages"], s["k_scales"],
                                    s["v_scales"], phases=s["phases"], layout=c["layout"], mscale=s["mscale"],
                                    k_weight=s["wk"], q_weight=s["wq"], eps=_EPS, q=s["q"], q_out=s["q_out"])
            k, v = blkattn.paged_read_q8(s["look"], s["table"], s["k_pages"], s["v_pages"], s["k_scales"],
                                         s["v_scales"])
            return k, v, s["q_out"]
        if c["op"] == "read":
            return blkattn.paged_read_q8(s["look"], s["table"], s["k_pages"], s["v_pages"], s["k_scales"],
                                         s["v_scales"], out_dtype=_DT[c["out"]])
        return blkattn.attention_paged_q8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                                          s["lens"], s["pos"], out_dtype=_DT[c["out"]], tree=s["tree"],
                                          window=c["window"])
    if c["op"] == "norm":
        return tuple(_rotate(s, _normed(s[x], s["w" + x])).to(_DT[c["out"]]) for x in "qk")
    if c["op"] == "norm_bwd":
        dq, dwq = _norm_gradient(s, s["gq"], s["q"], s["wq"], _DT[c["out"]])
        dk, dwk = _norm_gradient(s, s["gk"], s["k"], s["wk"], _DT[c["out"]])
        return dq, dk, dwq, dwk
    if c["op"] == "append":
        k, q = (_rotate(s, _normed(s[x], s["w" + x])) for x in "kq")
        _written(s, k, s["k_pages"], s["k_scales"])
        _written(s, s["v"].float(), s["v_pages"], s["v_scales"])
        s["q_out"].copy_(torch.where((s["pos"] >= 0)[:, None, :, None], q, 0.0))
        return (*(_look(s, s[x + "_pages"], s[x + "_scales"], torch.bfloat16) for x in "kv"), s["q_out"])
    if c["op"] == "read":
        return tuple(_look(s, s[x + "_pages"], s[x + "_scales"], _DT[c["out"]]) for x in "kv")
    return _plain_attend(s)


def _visible(case):
    """(visible (row, key) pairs of one query head, cache rows read), over all sequences."""
    T, w = case["T"], case["window"]
    lens = _spread(case["lo"], case["hi"], case["B"])
    pairs = rows = 0
    for n in lens:
        first = n - T + 1 if case["kind"] == "causal" else n
        ends = [min(n, first + i) for i in range(T)] if case["kind"] == "causal" else [n] * T
        pairs += sum(min(e, w) if w else e for e in ends)
        rows += min(n, w + T - 1) if w else n
    return pairs, rows


def work(case):
    B, T, d, Hkv = case["B"], case["T"], case["d"], case["Hkv"]
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    o = 2 if case.get("out", "bf16") == "bf16" else 4
    if case["op"] in ("norm", "norm_bwd"):
        n = B * (case["Hq"] + Hkv) * T
        if case["op"] == "norm":
            return {"bytes": n * d * (e + o) + 4 * B * T, "flops": n * (4.0 * d + 3.0 * case["rot"])}
        return {"bytes": n * d * (4 + e + o) + 4 * B * T + 8 * d, "flops": n * (12.0 * d + 3.0 * case["rot"])}
    cell = d + 1.0 / case["S"]  # bytes of a cache row
    if case["op"] == "append":
        n = sum(_spread(max(1, T // 4), T, B)) if case["ragged"] else B * T
        # the new rows and queries in and out, and the blocks read back (their numbers and what they stand for)
        return {"bytes": n * (2 * Hkv * (d * e + cell) + 2 * case["Hq"] * d * e) + 2 * n * Hkv * (cell + 2 * d) + 12 * B * T,
                "flops": n * (3.0 * case["rot"] + 4.0 * d * case["norm"]) * (Hkv + case["Hq"]) + 4.0 * n * Hkv * d}
    if case["op"] == "read":
        n = sum(_spread(case["lo"], case["hi"], B))
        return {"bytes": 2 * Hkv * (n * cell + B * T * d * o) + 4 * B * T, "flops": 2.0 * n * Hkv * d}
    pairs, rows = _visible(case)
    return {"bytes": 2 * rows * Hkv * cell + B * case["Hq"] * T * (d * (2 + o) + 4) + 4 * (rows // case["page"]),
            "flops": 4.0 * pairs * case["Hq"] * d}


# --------------------------------------------------------- 64-bit answers
def _turned(s, x):
    """The rows' rotation as products of complex numbers, in 64 bits."""
    rot = s["case"]["rot"]
    if rot == 0:
        return x
    part = x[..., :rot]
    half = s["case"]["layout"] == "half"
    pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if half else part.unflatten(-1, (rot // 2, 2))
    angle = s["pos"].double()[:, None, :, None] * s["w"]
    z = torch.complex(pairs[..., 0], pairs[..., 1]) * torch.polar(torch.full_like(angle, s["mscale"]), angle)
    both = (z.real, z.imag)
    y = torch.cat(both, -1) if half else torch.stack(both, -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _head_norm(x, w):
    """x / its root mean square, times w, in 64 bits."""
    return x if w is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w


def _to_grid(x, e):
    """x in 64 bits rounded to the nearest number that e4m3 times 2^e can hold (ties to even; x is within range)."""
    u = x * torch.exp2(-e)
    k = torch.frexp(u).exponent.clamp(min=-5).double() - 4  # 2^k: the step at u
    return torch.where(torch.isfinite(x), torch.round(u * torch.exp2(-k)) * torch.exp2(k + e), math.nan)


def _cache_rows(s, name, b, h, n):
    """The first n cache rows of a sequence and head in 64 bits, [n, d]."""
    P, S = s["case"]["page"], s["case"]["S"]
    ids = s["table"][b, : -(-n // P)].long()
    x = s[name + "_pages"][ids, h].double()
    e = s[name + "_scales"].view(torch.uint8)[ids, h].double() - 127
    return (x * torch.exp2(e).repeat_interleave(S, 1)[..., None]).flatten(0, 1)[:n], e.repeat_interleave(S, 1).flatten()[:n]


def _exact_append(s):
    c = s["case"]
    S, B, T, H, d = (c[k] for k in ("S", "B", "T", "Hkv", "d"))
    W = s["look"].shape[1]
    found = [torch.zeros((B, H, W, d), dtype=torch.float64, device="cuda") for _ in range(2)]
    k, q = (_turned(s, _head_norm(s[x].double(), None if s["w" + x] is None else s["w" + x].double())) for x in "kq")
    for b, p in enumerate(s["pos"].tolist()):
        n = sum(x >= 0 for x in p)
        end = p[0] + n
        for h in range(H):
            for out, name, new in zip(found, "kv", (k, s["v"].double())):
                rows, e_old = _cache_rows(s, name, b, h, -(-end // S) * S)
                rows[p[0]:end] = new[b, h, :n]
                base = p[0] // S * S
                blocks = torch.arange(base, end, device="cuda") // S
                size = torch.zeros(int(blocks[-1]) + 1, dtype=torch.float64, device="cuda")
                size.index_reduce_(0, blocks[p[0] - base:], rows[p[0]:end].abs().amax(1), "amax")
                m, ex = torch.frexp(size)
                e = torch.where(size == 0, -127, ex - 9 + (m > 0.875)).clamp(min=-127)
                e = e.repeat_interleave(S)[base:end].double()
                if base < p[0]:  # the block went on: its exponent does not fall
                    e[:S] = torch.maximum(e[:S], e_old[base:base + S][: e[:S].shape[0]])
                out[b, h, : end - base] = _to_grid(rows[base:end], e[:, None])
    q = torch.where((s["pos"] >= 0)[:, None, :, None], q, 0.0)
    return found[0], found[1], q


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return tuple(_turned(s, _head_norm(s[x].double(), s["w" + x].double())) for x in "qk")
    if c["op"] == "norm_bwd":
        dx, dw = [], []
        for x in "qk":
            w = s["w" + x].double().requires_grad_()
            dx.append(torch.empty(s[x].shape, dtype=torch.float64, device="cuda"))
            for h in range(s[x].shape[1]):
                leaf = s[x][:, h:h + 1].double().requires_grad_()
                _turned(s, _head_norm(leaf, w)).backward(s["g" + x][:, h:h + 1].double())
                dx[-1][:, h:h + 1] = leaf.grad
            dw.append(w.grad)
        return (*dx, *dw)
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "read":
        out = [torch.zeros((c["B"], c["Hkv"], c["T"], c["d"]), dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, n in enumerate(s["lens"].tolist()):
            for h in range(c["Hkv"]):
                for x, name in zip(out, "kv"):
                    x[b, h, :n] = _cache_rows(s, name, b, h, n)[0]
        return tuple(out)
    B, T, Hq, Hkv, d = (c[k] for k in ("B", "T", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    out = torch.zeros((B, Hq, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        pos = s["pos"][b].long()
        j = torch.arange(n, device="cuda")
        hide = j[None, :] > pos[:, None]
        if c["window"]:
            hide |= j[None, :] <= (pos - c["window"])[:, None]
        if s["tree"] is not None:
            inside = torch.arange(T, device="cuda")
            hide[:, n - T:] |= ((s["tree"][b][:, None] >> inside[None, :]) & 1) == 0
        for h in range(Hkv):
            k, v = (_cache_rows(s, x, b, h, n)[0] for x in "kv")
            for i in range(h * G, (h + 1) * G):
                z = (s["q"][b, i].double() @ k.T) / math.sqrt(d)
                z = z.masked_fill(hide, -math.inf)
                a = torch.logsumexp(z, dim=1)
                seen = a > -math.inf
                lse[b, i] = a
                out[b, i][seen] = torch.softmax(z[seen], dim=1) @ v
    return out, lse
