"""Measured cases of the rotary, paged-append and paged-attention operators.

Every case names one operator and its sizes.  `run` computes it either in its
plain form (elementary torch operations) or, with `own`, through the library's
binding.  Shapes are the library's: rows [B, heads, T, d], pools
[pages, KV heads, page rows, d], page tables int32 [B, entries].

Positions are turned into angles by a table of phases: F_i = round(2^64 w_i /
2 pi), the turn per position as a 64-bit fraction, so that a far position's
angle wraps exactly.  The plain form takes the angles w_i in 64 bits.
"""
import math
from fractions import Fraction

import numpy as np
import torch

own = False

_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _rope(name, B, H, T, d, rot, layout="half", dtype="bf16", out="bf16", bwd=False, first=0, scaled=False,
          token_major=True):
    return {"name": name, "op": "rope", "B": B, "H": H, "T": T, "d": d, "rot": rot, "layout": layout,
            "dtype": dtype, "out": out, "bwd": bwd, "first": first, "scaled": scaled, "token_major": token_major}


def _append(name, B, Hq, Hkv, T, d, rot, page, lo, hi, layout="half", dtype="bf16", rows_major=False, ragged=False):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "rot": rot, "page": page,
            "lo": lo, "hi": hi, "layout": layout, "dtype": dtype, "rows_major": rows_major, "ragged": ragged}


def _attend(name, B, Hq, Hkv, T, d, page, lo, hi, kind="causal", window=0, dtype="bf16", rows_major=False,
            absent=0):
    return {"name": name, "op": "attend", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "page": page, "lo": lo,
            "hi": hi, "kind": kind, "window": window, "dtype": dtype, "rows_major": rows_major, "absent": absent}


def listed():
    return [
        # the query rows of one decode step of 32 sequences: the smallest call, latency counts
        _rope("rope_decode_step", 32, 32, 1, 128, 128, first=8000),
        # the query rows of a whole prompt, as a projection lays them out (token-major)
        _rope("rope_prompt", 2, 32, 8192, 128, 128),
        # the backward pass: f32 dq as the attention's backward writes it, to bf16 for the projection's gradient
        _rope("rope_bwd_prompt", 2, 32, 8192, 128, 128, dtype="f32", out="bf16", bwd=True, token_major=False),
        # odd sizes, part of the head, interleaved pairs, far scaled positions, 32-bit gradients
        _rope("rope_bwd_far_part", 3, 5, 1777, 64, 24, layout="interleaved", dtype="f32", out="f32", bwd=True,
              first=1000000, scaled=True),
        # one decode step of 32 sequences into small pages, with its query rows
        _append("append_decode_step", 32, 32, 8, 1, 128, 128, 16, 512, 8191),
        # a chunk of prompts of different lengths (short ones padded), pages of 64
        _append("append_prompt_chunk", 4, 64, 8, 2048, 128, 128, 64, 0, 2048, ragged=True),
        # batched decode over small pages
        _attend("decode_batch_p16", 32, 32, 8, 1, 128, 16, 512, 8192),
        # one long context, one page a tile
        _attend("decode_long_p128", 1, 32, 8, 1, 128, 128, 131072, 131072, rows_major=True),
        # verification of six-node token trees, some nodes absent
        _attend("verify_tree_p32", 8, 64, 8, 6, 128, 32, 1024, 32768, kind="tree", absent=2),
        # the last 2048 rows of prompts, over the pages that hold all of them
        _attend("prompt_chunk_p64", 2, 32, 8, 2048, 128, 64, 8192, 8192),
        # heads of 64 under a sliding window
        _attend("decode_window_d64", 16, 64, 8, 1, 64, 16, 8192, 16384, window=4096),
        # one 32-bit row: the smallest attention call
        _attend("decode_tiny_f32", 1, 1, 1, 1, 64, 16, 1000, 1000, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "append", "attend", "attend", "attend"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    d = rng.choice((64, 128))
    if op == "rope":
        T, H = _log(rng, 1, 8192), _log(rng, 1, 64)
        B = max(1, min(_log(rng, 1, 64), (1 << 18) // (T * H)))
        return {k: v for k, v in _rope("", B, H, T, d, rng.choice((d, d, d // 2, 2 * rng.randint(1, d // 2))),
                                       layout=rng.choice(("half", "interleaved")), dtype=dtype,
                                       out=rng.choice(("bf16", "f32")), bwd=rng.random() < 0.5,
                                       first=_log(rng, 1, 1 << 21), scaled=rng.random() < 0.5,
                                       token_major=rng.random() < 0.5).items() if k != "name"}
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 7, 8))
    page = rng.choice((8, 16, 16, 32, 64, 128, 256))
    rows_major = rng.random() < 0.5
    if op == "append":
        T = _log(rng, 1, 2048)
        B = max(1, min(_log(rng, 1, 64), 2048 // T))
        lo = _log(rng, 1, 4096)
        return {k: v for k, v in _append("", B, G * Hkv, Hkv, T, d, rng.choice((0, d, d, d // 2)), page, lo,
                                         lo + rng.randint(0, 2048), layout=rng.choice(("half", "interleaved")),
                                         dtype=dtype, rows_major=rows_major,
                                         ragged=rng.random() < 0.5).items() if k != "name"}
    kind = rng.choice(("causal", "causal", "tree", "window"))
    if kind != "tree" and dtype == "bf16" and d == 128 and rng.random() < 0.35:
        T, B = _log(rng, 64, 2048), 1 if G * Hkv > 32 else rng.randint(1, 2)  # a prompt's chunk
        hi = _log(rng, T, 8192)
        lo = rng.randint(T, hi)
    else:
        T, B = rng.choice((1, 1, 2, 5, 8, 17)), _log(rng, 1, 32)
        hi = _log(rng, max(T, 16), 131072 // B)
        lo = rng.randint(max(T, hi // 8), hi)
        if dtype == "f32":  # the 32-bit kernel serves small work
            hi, lo = max(T, hi // 8), max(T, lo // 8)
    window = _log(rng, 1, hi) if kind == "window" else 0
    return {k: v for k, v in _attend("", B, G * Hkv, Hkv, T, d, page, lo, hi,
                                     kind="tree" if kind == "tree" else "causal", window=window, dtype=dtype,
                                     rows_major=rows_major,
                                     absent=rng.randint(0, max(0, min(T - 1, 3)))).items() if k != "name"}


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
    """Page tables whose pages lie in random order in a pool with a few spare pages; entries past a sequence's pages are -1."""
    need = [-(-n // page) for n in lens]
    N = sum(need) + spare
    order = _order(g, N).to(torch.int32)
    table = torch.full((len(lens), max(1, entries)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, N


def _pool(g, N, Hkv, page, d, dtype, rows_major):
    if rows_major:
        return _normal(g, (N, page, Hkv, d), dtype).transpose(1, 2)
    return _normal(g, (N, Hkv, page, d), dtype)


def _rows(g, B, H, T, d, dtype, token_major=True):
    """[B, H, T, d], stored token by token as a projection writes them."""
    return _normal(g, (B, T, H, d), dtype).transpose(1, 2) if token_major else _normal(g, (B, H, T, d), dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    B, T, d = case["B"], case["T"], case["d"]
    dtype = _DT[case["dtype"]]
    if case["op"] == "rope":
        w, s["mscale"] = _angles(case)
        s["w"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        s["phases"] = _phases(w)
        s["x"] = _rows(g, B, case["H"], T, d, dtype, case["token_major"])
        start = torch.randint(0, case["first"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        return s
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    perm = _order(g, B).tolist()
    lens = [_spread(case["lo"], case["hi"], B)[i] for i in perm]
    if case["op"] == "append":
        w, s["mscale"] = _angles(case)
        s["w"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        s["phases"] = _phases(w) if w else None
        new = [_spread(max(1, T // 4), T, B)[i] for i in perm] if case["ragged"] else [T] * B
        s["table"], N = _tables(g, [n + T for n in lens], -(-(case["hi"] + T) // page), page, 3)
        s["k_pages"] = _pool(g, N, Hkv, page, d, dtype, case["rows_major"])
        s["v_pages"] = _pool(g, N, Hkv, page, d, dtype, case["rows_major"])
        s["k"], s["v"], s["q"] = (_rows(g, B, h, T, d, dtype) for h in (Hkv, Hkv, Hq))
        s["q_out"] = torch.zeros((B, Hq, T, d), dtype=dtype, device="cuda")
        t = torch.arange(T, device="cuda")
        first, n = (torch.tensor(v, device="cuda")[:, None] for v in (lens, new))
        s["pos"] = torch.where(t < n, first + t, -1).to(torch.int32)  # -1: a row that is padding
        return s
    s["table"], N = _tables(g, lens, -(-case["hi"] // page), page, 3)
    s["k_pages"] = _pool(g, N, Hkv, page, d, dtype, case["rows_major"])
    s["v_pages"] = _pool(g, N, Hkv, page, d, dtype, case["rows_major"])
    s["q"] = _rows(g, B, Hq, T, d, dtype)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    t = torch.arange(T, device="cuda")
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
def _rotate(x, pos, w, rot, layout, mscale, sign):
    """Rows x [B, H, T, d] rotated in 32 bits; the angles in 64 (32 bits lose those of far positions)."""
    if rot == 0:
        return x.float()
    a = sign * pos.double()[:, None, :, None] * w  # [B, 1, T, rot / 2]
    cos, sin = (torch.cos(a) * mscale).float(), (torch.sin(a) * mscale).float()
    y = x.float().clone()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., lo].float(), x[..., hi].float()
    y[..., lo] = u * cos - v * sin
    y[..., hi] = u * sin + v * cos
    return y


def _gathered(pages, table, page, T):
    """The cache rows of each sequence in order: [B, Hkv, T, d] in 32 bits (absent pages: page 0's rows, masked by the caller)."""
    B, n = table.shape
    x = pages[table.clamp(min=0).long()]  # [B, n, Hkv, page, d]
    return x.transpose(1, 2).reshape(B, x.shape[2], n * page, x.shape[4])[:, :, :T].float()


def _plain_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, d, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "page"))
    K = min(c["hi"], s["table"].shape[1] * page)
    k, v = (_gathered(s[n], s["table"], page, K) for n in ("k_pages", "v_pages"))
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
    return o.reshape(B, Hq, T, d).to(_DT[c["dtype"]]), lse


def run(s):
    c = s["case"]
    if own:
        from exact_blocked_attention_gb300 import blkattn
        if c["op"] == "rope":
            f = blkattn.rope_backward if c["bwd"] else blkattn.rope
            return f(s["x"], s["pos"], s["phases"], layout=c["layout"], mscale=s["mscale"], out_dtype=_DT[c["out"]])
        if c["op"] == "append":
            blkattn.paged_append(s["k"], s["v"], s["pos"], s["table"], s["k_pages"], s["v_pages"],
                                 phases=s["phases"], layout=c["layout"], mscale=s["mscale"], q=s["q"],
                                 q_out=s["q_out"])
            return s["k_pages"], s["v_pages"], s["q_out"]
        return blkattn.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["pos"],
                                       out_dtype=_DT[c["dtype"]], tree=s["tree"], window=c["window"])
    if c["op"] == "rope":
        y = _rotate(s["x"], s["pos"], s["w"], c["rot"], c["layout"], s["mscale"], -1 if c["bwd"] else 1)
        return y.to(_DT[c["out"]])
    if c["op"] == "append":
        k, q = (_rotate(s[n], s["pos"], s["w"], c["rot"], c["layout"], s["mscale"], 1).to(s[n].dtype) for n in "kq")
        if c["ragged"]:
            b, i = torch.nonzero(s["pos"] >= 0, as_tuple=True)
        else:
            b, i = (x.reshape(-1) for x in torch.meshgrid(torch.arange(c["B"], device="cuda"),
                                                          torch.arange(c["T"], device="cuda"), indexing="ij"))
        t = s["pos"][b, i].long()
        page = s["table"][b, t // c["page"]].long()
        s["k_pages"][page, :, t % c["page"]] = k[b, :, i]
        s["v_pages"][page, :, t % c["page"]] = s["v"][b, :, i]
        s["q_out"][b, :, i] = q[b, :, i]
        return s["k_pages"], s["v_pages"], s["q_out"]
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
    B, T, d = case["B"], case["T"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = B * case["H"] * T
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": n * d * (e + o) + 4 * B * T, "flops": 3.0 * n * case["rot"]}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "append":
        rows = sum(_spread(max(1, T // 4), T, B)) if case["ragged"] else B * T
        return {"bytes": 2 * rows * (Hq + 2 * Hkv) * d * e + 8 * B * T, "flops": 3.0 * rows * (Hq + Hkv) * case["rot"]}
    pairs, rows = _visible(case)
    return {"bytes": 2 * rows * Hkv * d * e + B * Hq * T * (2 * d * e + 4) + 4 * (rows // case["page"]),
            "flops": 4.0 * pairs * Hq * d}


# --------------------------------------------------------- 64-bit answers
def _turned(x, pos, w, rot, layout, mscale, sign):
    """The rows' rotation as products of complex numbers, in 64 bits."""
    y = x.double().clone()
    if rot == 0:
        return y
    part = y[..., :rot]
    pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if layout == "half" else part.unflatten(-1, (rot // 2, 2))
    angle = sign * pos.double()[:, None, :, None] * w
    z = torch.complex(pairs[..., 0], pairs[..., 1]) * torch.polar(torch.full_like(angle, mscale), angle)
    both = (z.real, z.imag)
    y[..., :rot] = torch.cat(both, -1) if layout == "half" else torch.stack(both, -1).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _turned(s["x"], s["pos"], s["w"], c["rot"], c["layout"], s["mscale"], -1 if c["bwd"] else 1)
    if c["op"] == "append":
        kp, vp, qo = (s[n].double().contiguous() for n in ("k_pages", "v_pages", "q_out"))
        k, q = (_turned(s[n], s["pos"], s["w"], c["rot"], c["layout"], s["mscale"], 1) for n in "kq")
        v = s["v"].double()
        pos, table = s["pos"].cpu().numpy(), s["table"].cpu().numpy()
        for b in range(c["B"]):
            rows = np.flatnonzero(pos[b] >= 0)
            for p in np.unique(pos[b][rows] // c["page"]):  # one page of one sequence at a time
                i = rows[pos[b][rows] // c["page"] == p]
                at = torch.from_numpy(pos[b][i] % c["page"]).long().cuda()
                i = torch.from_numpy(i).cuda()
                kp[int(table[b, p])][:, at] = k[b][:, i]
                vp[int(table[b, p])][:, at] = v[b][:, i]
            i = torch.from_numpy(rows).cuda()
            qo[b][:, i] = q[b][:, i]
        return kp, vp, qo
    B, T, Hq, Hkv, d, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "page"))
    G = Hq // Hkv
    out = torch.zeros((B, Hq, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        ids = s["table"][b, : -(-n // page)].long()
        pos = s["pos"][b].long()
        tree = s["tree"][b] if s["tree"] is not None else None
        j = torch.arange(n, device="cuda")
        for h in range(Hkv):
            k = s["k_pages"][ids, h].double().reshape(-1, d)[:n]
            v = s["v_pages"][ids, h].double().reshape(-1, d)[:n]
            hide = j[None, :] > pos[:, None]
            if c["window"]:
                hide |= j[None, :] <= (pos - c["window"])[:, None]
            if tree is not None:
                inside = torch.arange(T, device="cuda")
                hide[:, n - T:] |= ((tree[:, None] >> inside[None, :]) & 1) == 0
            for g in range(G):
                z = (s["q"][b, h * G + g].double() @ k.T) / math.sqrt(d)
                z = z.masked_fill(hide, -math.inf)
                a = torch.logsumexp(z, dim=1)
                seen = a > -math.inf
                lse[b, h * G + g] = a
                out[b, h * G + g][seen] = torch.softmax(z[seen], dim=1) @ v
    return out, lse
