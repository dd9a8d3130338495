"""Cases of the serving operators around rotary positions and latent attention, in plain torch
operations and as the framework's calls.

Rotary positions: the first 2 h channels of a head are turned in h pairs, pair i of the token at
position p by the angle p * w_i: (a, b) -> (a cos - b sin, b cos + a sin).  The pairs are channels
(i, i + h) (half) or (2 i, 2 i + 1) (interleaved).  A table [positions, 2 h] in fp32 holds the
cosines, then the sines, both times a factor that long-context scaling of the w_i brings along.
Tokens of padding have position -1 (they are not turned) and slot -1 (they are not stored).

  rotary   queries and keys of a step turned, or turned back (the gradient of that)
  append   the same on the way of new keys into a paged key/value cache held in 8 bits (pages of P
           tokens, codes e4m3, one power-of-two scale per page and head that grows when a larger
           value arrives, the page's older codes then rounded again); queries are turned beside it
  store    a token's shared latent vector (C channels) and its turned key part (R channels) into
           a paged cache [pages, P, C + R] in 16 bits; the queries' R channels are turned beside it
  absorbed attention whose keys are the C + R channels of such a cache and whose values are their
           first C: the key and value projections are absorbed into the queries and the output
  expanded the same attention of whole prompts with keys and values laid out per head again: keys
           of Dn channels and R more that all heads share, values of Dv channels; requests ragged
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_E4M3 = torch.float8_e4m3fn
_E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the queries and keys of one decode step of a small batch, far into their contexts
        {"name": "rotary, decode step", "op": "rotary", "T": 8, "Hq": 32, "Hk": 8, "d": 128, "rot": 128,
         "pairs": "half", "back": False, "at": 100000, "scaled": 8.0, "dtype": "bf16"},
        # the tokens of several prompts at once
        {"name": "rotary, prompts", "op": "rotary", "T": 16000, "Hq": 32, "Hk": 8, "d": 128, "rot": 128,
         "pairs": "half", "back": False, "at": 0, "scaled": 1.0, "dtype": "bf16"},
        # the gradient of a part of odd head counts that is turned in neighbouring pairs
        {"name": "rotary, gradient", "op": "rotary", "T": 4001, "Hq": 15, "Hk": 5, "d": 96, "rot": 64,
         "pairs": "interleaved", "back": True, "at": 777, "scaled": 4.0, "dtype": "fp16"},
        # the tokens of one decode step
        {"name": "append, decode step", "op": "append", "B": 32, "Hq": 32, "Hk": 8, "d": 128, "rot": 128, "P": 64,
         "len": 4096, "new": 1, "pairs": "half", "scaled": 1.0, "dtype": "bf16", "bounds": True},
        # whole prompts written at once
        {"name": "append, prompts", "op": "append", "B": 8, "Hq": 32, "Hk": 8, "d": 128, "rot": 64, "P": 64,
         "len": 0, "new": 4096, "pairs": "interleaved", "scaled": 4.0, "dtype": "bf16", "bounds": False},
        # the latent vectors of one decode step
        {"name": "store, decode step", "op": "store", "B": 64, "H": 128, "C": 512, "R": 64, "P": 64,
         "len": 5000, "new": 1, "pairs": "interleaved", "scaled": 40.0, "dtype": "bf16"},
        # the latent vectors of prompts
        {"name": "store, prompts", "op": "store", "B": 5, "H": 16, "C": 512, "R": 64, "P": 32,
         "len": 100, "new": 5000, "pairs": "half", "scaled": 1.0, "dtype": "bf16"},
        # one user's next token after a context of 4096
        {"name": "absorbed, one request", "op": "absorbed", "B": 1, "H": 32, "C": 512, "R": 64, "P": 64,
         "len": 4096, "new": 1, "dtype": "bf16"},
        # the next tokens of a ragged batch with contexts up to 16384
        {"name": "absorbed, ragged batch", "op": "absorbed", "B": 64, "H": 128, "C": 512, "R": 64, "P": 64,
         "len": 16384, "new": 1, "dtype": "bf16"},
        # drafts of a few tokens that are checked together; odd head count, short latents, small pages
        {"name": "absorbed, drafts", "op": "absorbed", "B": 7, "H": 20, "C": 256, "R": 32, "P": 16,
         "len": 6001, "new": 5, "dtype": "fp16"},
        # pieces of long prompts against what came before them
        {"name": "expanded, prompt pieces", "op": "expanded", "B": 2, "H": 32, "Dn": 128, "R": 64, "Dv": 128,
         "len": 6000, "new": 4000, "dtype": "bf16"},
        # short ragged prompts with odd head count and widths
        {"name": "expanded, short prompts", "op": "expanded", "B": 9, "H": 5, "Dn": 96, "R": 32, "Dv": 80,
         "len": 333, "new": 333, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "store", "absorbed", "absorbed", "expanded"])
    dtype = rng.choice(["bf16", "fp16"])
    turn = {"pairs": rng.choice(["half", "interleaved"]), "scaled": rng.choice([1.0, 4.0, 40.0])}
    P = rng.choice([16, 32, 64, 128])
    if op in ("rotary", "append"):
        Hk, G = rng.choice([1, 2, 3, 5, 8]), rng.choice([1, 2, 3, 4, 5])
        d = rng.choice([64, 80, 96, 128, 256])
        heads = {"Hq": Hk * G, "Hk": Hk, "d": d, "rot": rng.choice([d, d, 16, d // 2 if d % 32 == 0 else d])}
        if op == "rotary":
            return {"op": op, "T": _log(rng, 1, 8000), **heads, "back": rng.random() < 0.4,
                    "at": rng.choice([0, _log(rng, 1, 100000)]), **turn, "dtype": dtype}
        one = rng.random() < 0.5
        return {"op": op, "B": _log(rng, 1, 256) if one else _log(rng, 1, 8), **heads, "P": P,
                "len": _log(rng, 1, 2000) if one else rng.choice([0, _log(rng, 1, 500)]),
                "new": 1 if one else _log(rng, 2, 2500), **turn, "dtype": dtype, "bounds": rng.random() < 0.5}
    H = rng.choice([1, 3, 5, 8, 16])
    if op == "expanded":
        Dn, R, Dv = rng.choice([(128, 64, 128), (64, 32, 64), (96, 32, 80), (128, 64, 64), (48, 16, 112)])
        new = _log(rng, 1, 2600)
        return {"op": op, "B": rng.randint(1, 4), "H": H, "Dn": Dn, "R": R, "Dv": Dv,
                "len": new + rng.choice([0, _log(rng, 1, 2000)]), "new": new, "dtype": dtype}
    C, R = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32), (128, 32), (320, 16)])
    c = {"op": op, "B": _log(rng, 1, 40), "H": rng.choice([H, 16, 20, 32, 64, 128]), "C": C, "R": R, "P": P}
    if op == "store":
        one = rng.random() < 0.5
        return {**c, "len": _log(rng, 1, 4000), "new": 1 if one else _log(rng, 2, 1000), **turn, "dtype": dtype}
    return {**c, "len": _log(rng, 1, 10000), "new": 1 if rng.random() < 0.6 else rng.randint(2, 6), "dtype": dtype}


def _spread(n, top, low):
    """n whole numbers in [low * top, top], ragged, the first one `top`."""
    f = (np.arange(n) * 0.6180339887498949) % 1.0
    return np.maximum(1, np.floor(top * (1.0 - (1.0 - low) * f))).astype(np.int64)


def _sizes(c):
    """(tokens before the step, new tokens) of each request.  "len" counts the new tokens too for attention."""
    B = c["B"]
    lens = _spread(B, c["len"], 0.3) if c["len"] else np.zeros(B, np.int64)
    new = _spread(B, c["new"], 0.4)
    if c["op"] in ("absorbed", "expanded"):
        new = np.minimum(new, lens)
        lens = lens - new
    return lens, new


def _pages(n, P):
    return -(-n // P)


# --------------------------------------------------------------- inputs
def _frequencies(rot, scaled):
    """w_i = 10000^(-2 i / rot).  Scaled by s for contexts longer than 4096: pairs that turn fewer than once
    in 4096 positions are slowed by s, those of more than 32 turns are not, between them by a ramp over i; with it comes a factor."""
    h = rot // 2
    i = np.arange(h, dtype=np.float64)
    w = 10000.0 ** (-2.0 * i / rot)
    if scaled == 1.0:
        return w, 1.0
    at = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    keep = 1.0 - np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
    return w / scaled * (1.0 - keep) + w * keep, 0.1 * math.log(scaled) + 1.0


def _table(n, rot, scaled):
    w, factor = _frequencies(rot, scaled)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * torch.as_tensor(w, device="cuda")
    return torch.cat([torch.cos(a) * factor, torch.sin(a) * factor], dim=1).float()


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _scale_of(amax):
    """Smallest power of two s in [2^-60, 2^60] with amax <= 448 s (s = 2^60 where none is)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), e)


def _round_e4m3(x):
    return x.clamp(-_E4M3_MAX, _E4M3_MAX).to(_E4M3)  # NaN stays NaN


def _random_codes(g, pages, Hk, P, d):
    """Codes and scales of pages of keys or values whose size differs by page and head."""
    x = torch.randn((pages, Hk, P, d), device="cuda", generator=g)
    x *= torch.exp(0.4 * torch.randn((pages, Hk, 1, 1), device="cuda", generator=g))
    s = _scale_of(x.abs().amax(dim=(2, 3)))
    return _round_e4m3(x / s[:, :, None, None]), s


def _bounds_of(codes, filled):
    """Per page, head and channel: floor and ceil of (least, largest code) / 4 over the filled
    places, as [pages, Hk, 2, d] int8."""
    x = codes.float().nan_to_num(nan=0.0)
    at = (torch.arange(x.shape[2], device=x.device)[None, :] < filled[:, None])[:, None, :, None]
    lo = torch.where(at, x, torch.full_like(x, math.inf)).amin(dim=2)
    hi = torch.where(at, x, torch.full_like(x, -math.inf)).amax(dim=2)
    return torch.stack([torch.floor(lo / 4), torch.ceil(hi / 4)], dim=2).to(torch.int8)


def _paged(g, held, spare):
    """(block table, pages in all) of requests that hold these counts of pages, in shuffled order."""
    B, M, pool = len(held), int(held.max()), int(held.sum()) + spare
    table = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    col = torch.arange(M, device="cuda")[None, :] < torch.as_tensor(held, device="cuda")[:, None]
    table[col] = torch.randperm(pool, device="cuda", generator=g)[:int(held.sum())].to(torch.int32)
    return table, col, pool


def _step(c, table, before, new, padding):
    """Slots and positions of a step's tokens, some rows of padding behind them."""
    P = c["P"]
    req = torch.as_tensor(np.repeat(np.arange(c["B"]), new), device="cuda")
    pos = torch.as_tensor(np.concatenate([np.arange(a, a + n) for a, n in zip(before, new)]), device="cuda")
    slots = table[req, pos // P].long() * P + pos % P
    none = torch.full((padding,), -1, device="cuda")
    return torch.cat([slots, none]).to(torch.int32), torch.cat([pos, none]).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    dt = _TYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    if c["op"] == "rotary":
        # projections come as one tensor [T, Hq + 2 Hk, d] of queries, keys and values
        qkv = randn(c["T"], c["Hq"] + 2 * c["Hk"], c["d"]).to(dt)
        at = torch.randint(0, c["at"] + 1, (1,), device="cuda", generator=g) if c["T"] > 64 else \
            torch.randint(0, c["at"] + 1, (c["T"],), device="cuda", generator=g)
        pos = (at + torch.arange(c["T"], device="cuda")).to(torch.int32)
        return {"case": c, "q": qkv[:, :c["Hq"]], "k": qkv[:, c["Hq"]:c["Hq"] + c["Hk"]], "positions": pos,
                "turn": _table(c["at"] + c["T"], c["rot"], c["scaled"])}
    before, new = _sizes(c)
    after, T = before + new, int(new.sum())
    if c["op"] == "expanded":
        H, Dn, R, Dv = c["H"], c["Dn"], c["R"], c["Dv"]
        keys = int(after.sum())
        # per head, keys and values come side by side from one projection of the latents
        kv = randn(keys, H, Dn + Dv).to(dt)
        return {"case": c, "q": randn(T, H, Dn + R).to(dt), "k": kv[..., :Dn], "v": kv[..., Dn:],
                "k_shared": randn(keys, R).to(dt), "cu_q": _i32(np.concatenate([[0], np.cumsum(new)])),
                "cu_k": _i32(np.concatenate([[0], np.cumsum(after)])), "max_q": int(new.max()),
                "max_k": int(after.max()), "scale": 1.0 / math.sqrt(Dn + R)}
    table, col, pool = _paged(g, _pages(after, c["P"]), 7)
    s = {"case": c, "table": table}
    if c["op"] == "absorbed":
        C, R = c["C"], c["R"]
        s["cache"] = randn(pool, c["P"], C + R).to(dt)
        s["q"] = randn(T, c["H"], C + R).to(dt)
        s["lens"] = _i32(after)
        s["cu_q"] = _i32(np.concatenate([[0], np.cumsum(new)])) if c["new"] > 1 else None
        s["max_q"] = int(new.max())
        s["scale"] = 1.0 / math.sqrt(128 + R)
        return s
    s["slots"], s["positions"] = _step(c, table, before, new, 2)
    if c["op"] == "store":
        C, R = c["C"], c["R"]
        # latents and key parts come from one projection, the queries' part from another
        kv = randn(T + 2, C + R).to(dt)
        s["latent"], s["k"] = kv[:, :C], kv[:, C:]
        s["q"] = randn(T + 2, c["H"], 128 + R).to(dt)[..., 128:]
        s["cache"] = randn(pool, c["P"], C + R).to(dt)
        s["turn"] = _table(int(after.max()), R, c["scaled"])
        return s
    Hq, Hk, d, P = c["Hq"], c["Hk"], c["d"], c["P"]
    s["k_cache"], s["k_scale"] = _random_codes(g, pool, Hk, P, d)
    s["v_cache"], s["v_scale"] = _random_codes(g, pool, Hk, P, d)
    qkv = randn(T + 2, Hq + 2 * Hk, d)
    qkv *= torch.exp(0.4 * randn(T + 2, Hq + 2 * Hk, 1))
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    s["turn"] = _table(int(after.max()), c["rot"], c["scaled"])
    s["bounds"] = None
    if c["bounds"]:
        filled = torch.ones(pool, dtype=torch.int64, device="cuda")
        j = torch.arange(table.shape[1], device="cuda")[None, :]
        held = (torch.as_tensor(before, device="cuda")[:, None] - j * P).clamp(1, P)
        filled[table[col].long()] = held[col]
        s["bounds"] = _bounds_of(s["k_cache"], filled)
    return s


# --------------------------------------------------------- the plain forms
def _turn(x, positions, table, pairs, back):
    """x [T, heads, d] in fp32 with its first table.shape[1] channels turned."""
    h = table.shape[1] // 2
    row = table[positions.clamp(min=0).long()][:, None]
    cos, sin = row[..., :h], row[..., h:]
    if back:
        sin = -sin
    if pairs == "half":
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    y = torch.cat([y, x[..., 2 * h:]], dim=-1)
    return torch.where((positions >= 0)[:, None, None], y, x)


def _plain_rotary(s):
    c = s["case"]
    q = _turn(s["q"].float(), s["positions"], s["turn"], c["pairs"], c["back"])
    k = _turn(s["k"].float(), s["positions"], s["turn"], c["pairs"], c["back"])
    return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype)}


def _quantise(x, slots, cache, scale):
    """Rows x [n, Hk, d] in fp32 into their slots; (pages written, their first and last place + 1)."""
    P = cache.shape[2]
    pages, at = torch.unique(slots // P, return_inverse=True)
    place = slots % P
    n, Hk = pages.numel(), x.shape[1]
    first = torch.full((n,), P, device=x.device).scatter_reduce(0, at, place, "amin")
    last = torch.zeros((n,), dtype=place.dtype, device=x.device).scatter_reduce(0, at, place + 1, "amax")
    amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(dim=2)
    amax = torch.zeros((n, Hk), device=x.device).scatter_reduce(0, at[:, None].expand(-1, Hk), amax, "amax")
    before = torch.where((first == 0)[:, None], 0.0, scale[pages])
    after = torch.maximum(before, _scale_of(amax))
    codes = cache[pages]
    old = codes.float() * torch.where(before > 0, before / after, 1.0)[:, :, None, None]
    older = torch.arange(P, device=x.device)[None, :] < first[:, None]
    codes = torch.where(older[:, None, :, None], _round_e4m3(old).view(torch.uint8), codes.view(torch.uint8))
    codes[at, :, place] = _round_e4m3(x / after[at][:, :, None]).view(torch.uint8)
    cache.view(torch.uint8)[pages] = codes
    scale[pages] = after
    return pages, last


def _plain_append(s):
    c = s["case"]
    keep = s["slots"] >= 0
    slots = s["slots"].long()[keep]
    q = _turn(s["q"].float(), s["positions"], s["turn"], c["pairs"], False)
    k = _turn(s["k"].float(), s["positions"], s["turn"], c["pairs"], False)
    pages, last = _quantise(k[keep], slots, s["k_cache"], s["k_scale"])
    _quantise(s["v"].float()[keep], slots, s["v_cache"], s["v_scale"])
    out = {"q": q.to(s["q"].dtype), "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if s["bounds"] is not None:
        s["bounds"][pages] = _bounds_of(s["k_cache"][pages], last)
        out["bounds"] = s["bounds"]
    return out


def _plain_store(s):
    c = s["case"]
    keep = s["slots"] >= 0
    k = _turn(s["k"].float()[:, None], s["positions"], s["turn"], c["pairs"], False)[:, 0]
    rows = torch.cat([s["latent"], k.to(s["k"].dtype)], dim=1)
    s["cache"].view(-1, c["C"] + c["R"])[s["slots"].long()[keep]] = rows[keep]
    q = _turn(s["q"].float(), s["positions"], s["turn"], c["pairs"], False)
    return {"cache": s["cache"], "q": q.to(s["q"].dtype)}


def _softmax_sum(x, v):
    """(weighted mean of v, log-sum-exp) over the last axis of scores x; rows that see nothing: 0, -inf."""
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _rows_of(cu, n):
    """(which of n places of each request are rows, their rows) as [B, n]."""
    i = torch.arange(n, device=cu.device)
    have = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    return have, torch.where(have, cu[:-1, None] + i, 0)


def _plain_absorbed(s):
    c = s["case"]
    B, H, C, n = c["B"], c["H"], c["C"], s["max_q"]
    lens = s["lens"].long()
    cu = s["cu_q"].long() if s["cu_q"] is not None else torch.arange(B + 1, device=lens.device)
    have, row = _rows_of(cu, n)
    q = s["q"].float()[row].view(B, n * H, -1)
    kv = s["cache"][s["table"].long()].float().view(B, -1, C + c["R"])    # [B, keys, C + R]
    x = torch.matmul(q, kv.transpose(1, 2)) * s["scale"]
    j = torch.arange(kv.shape[1], device=lens.device)
    last = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(n, device=lens.device)
    see = (j < lens[:, None, None]) & (j <= last[:, :, None])             # [B, n, keys]
    x = x.view(B, n, H, -1).masked_fill_(~see[:, :, None], -math.inf).view(B, n * H, -1)
    o, lse = _softmax_sum(x, kv[..., :C])
    return {"out": o.view(B, n, H, C)[have].to(s["q"].dtype), "lse": lse.view(B, n, H)[have]}


def _plain_expanded(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    have, row = _rows_of(cu_q, s["max_q"])
    there, key = _rows_of(cu_k, s["max_k"])
    q = s["q"].float()[row].transpose(1, 2)                               # [B, H, n, Dn + R]
    shared = s["k_shared"].float()[:, None].expand(-1, s["k"].shape[1], -1)
    k = torch.cat([s["k"].float(), shared], dim=-1)[key].transpose(1, 2)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device=q.device), torch.arange(s["max_k"], device=q.device)
    see = there[:, None, :] & (j[None, None, :] <= (nk - nq)[:, None, None] + i[None, :, None])
    o, lse = _softmax_sum(x.masked_fill_(~see[:, None], -math.inf), s["v"].float()[key].transpose(1, 2))
    return {"out": o.transpose(1, 2)[have].to(s["q"].dtype), "lse": lse.transpose(1, 2)[have]}


def _own(s):
    import online_softmax_tiling_gb300 as fa
    c = s["case"]
    if c["op"] == "rotary":
        q, k = fa.rotary_embed(s["q"], s["k"], s["positions"], s["turn"], interleaved=c["pairs"] == "interleaved",
                               inverse=c["back"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = fa.kv_cache_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["turn"], s["slots"], s["k_cache"],
                                      s["v_cache"], s["k_scale"], s["v_scale"], k_bounds=s["bounds"],
                                      interleaved=c["pairs"] == "interleaved")
        out = {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        return out if s["bounds"] is None else dict(out, bounds=s["bounds"])
    if c["op"] == "store":
        q = fa.latent_cache_append(s["latent"], s["k"], s["slots"], s["cache"], q_rope=s["q"], positions=s["positions"],
                                   table=s["turn"], interleaved=c["pairs"] == "interleaved")
        return {"cache": s["cache"], "q": q}
    if c["op"] == "absorbed":
        o, lse = fa.latent_paged_attention_forward(s["q"], s["cache"], s["table"], s["lens"], value_dim=c["C"],
                                                   cu_q=s["cu_q"], max_q=s["max_q"], scale=s["scale"])
        return {"out": o, "lse": lse}
    o, lse = fa.latent_attention_forward(s["q"], s["k"], s["k_shared"], s["v"], s["cu_q"], s["cu_k"], max_q=s["max_q"],
                                         max_k=s["max_k"], scale=s["scale"])
    return {"out": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "append": _plain_append, "store": _plain_store, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "rotary":
        # queries and keys read and written, a row of the table and a position per token
        return {"bytes": float(c["T"] * ((c["Hq"] + c["Hk"]) * c["d"] * 4 + c["rot"] * 4 + 4)),
                "flops": 3.0 * c["T"] * (c["Hq"] + c["Hk"]) * c["rot"]}
    before, new = _sizes(c)
    T = int(new.sum())
    if c["op"] == "append":
        P, Hk, d = c["P"], c["Hk"], c["d"]
        pages = int((_pages(before + new, P) - before // P).sum())
        b = T * (Hk * d * 2 * 2 + Hk * d * 2 + c["Hq"] * d * 4 + c["rot"] * 4 + 4) + 4 * (T + 2) + pages * Hk * 2 * 8
        if c["bounds"]:
            b += pages * Hk * 2 * d + int((before % P > 0).sum()) * Hk * 2 * d
        return {"bytes": float(b), "flops": 3.0 * T * (2 * Hk * d + (c["Hq"] + Hk) * c["rot"])}
    if c["op"] == "store":
        b = T * ((c["C"] + c["R"]) * 4 + c["H"] * c["R"] * 4 + c["R"] * 4 + 8)
        return {"bytes": float(b), "flops": 3.0 * T * (c["H"] + 1) * c["R"]}
    pairs = float((new * before + new * (new + 1) // 2).sum())  # of a query and a key it sees
    keys, H = float((before + new).sum()), c["H"]
    if c["op"] == "absorbed":
        C, W = c["C"], c["C"] + c["R"]
        b = keys * W * 2 + _pages(before + new, c["P"]).sum() * 4 + T * H * ((W + C) * 2 + 4)
        return {"bytes": float(b), "flops": 2.0 * pairs * H * (C + W)}
    Dk = c["Dn"] + c["R"]
    b = keys * (H * (c["Dn"] + c["Dv"]) + c["R"]) * 2 + T * H * ((Dk + c["Dv"]) * 2 + 4)
    return {"bytes": float(b), "flops": 2.0 * pairs * H * (Dk + c["Dv"])}


# ----------------------------------------- the definitions, in 64 bits
def _angles(s, rot, positions):
    """cos and sin [T, 1, h] of the tokens' angles (1 and 0 where there is no position), in 64 bits."""
    w, factor = _frequencies(rot, s["case"]["scaled"])
    p = positions.cpu().numpy().astype(np.float64)[:, None]
    cos, sin = np.where(p < 0, 1.0, np.cos(p * w) * factor), np.where(p < 0, 0.0, np.sin(p * w) * factor)
    return torch.as_tensor(cos, device="cuda")[:, None], torch.as_tensor(sin, device="cuda")[:, None]


def _turned(s, x, rot, back=False):
    cos, sin = _angles(s, rot, s["positions"])
    y = x.double().clone()
    h = rot // 2
    first, second = (slice(0, h), slice(h, rot)) if s["case"]["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cos, -sin if back else sin)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest_e4m3(x):
    """float64 -> the nearest e4m3 number (ties to even), at most 448 in size, as float64."""
    e = np.maximum(np.frexp(x)[1] - 1, -6)
    q = np.ldexp(1.0, e - 3)
    return np.clip(np.rint(x / q) * q, -448.0, 448.0)


def _exact_append(s):
    c, P = s["case"], s["case"]["P"]
    slots = s["slots"].cpu().numpy()
    runs, t = [], 0
    while t < len(slots):
        n = 1
        while slots[t] >= 0 and t + n < len(slots) and slots[t + n] // P == slots[t] // P:
            n += 1
        if slots[t] >= 0:
            runs.append((t, n, slots[t] // P, slots[t] % P))
        t += n
    out = {"q": _turned(s, s["q"], c["rot"])}
    for name, x in (("k", _turned(s, s["k"], c["rot"])), ("v", s["v"].double())):
        x = x.cpu().numpy()
        codes = s[name + "_cache"].float().cpu().numpy()
        scales = s[name + "_scale"].cpu().numpy().astype(np.float64)
        for t, n, page, place in runs:
            y = x[t:t + n].transpose(1, 0, 2)                             # [Hk, n, d]
            top = np.abs(y).max(axis=(1, 2))
            want = np.exp2(np.clip(np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -60, 60))
            now = want if place == 0 else np.maximum(want, scales[page])
            if place and (now > scales[page]).any():
                codes[page, :, :place] = _nearest_e4m3(codes[page, :, :place] * (scales[page] / now)[:, None, None])
            codes[page, :, place:place + n] = _nearest_e4m3(y / now[:, None, None])
            scales[page] = now
        out[name], out[name + "_scale"] = codes.astype(np.float64), scales
    if s["bounds"] is not None:
        out["bounds"] = None  # whole numbers of the codes as they were rounded from fp32
    return {k: out[k] for k in ("q", "k", "v", "k_scale", "v_scale", "bounds") if k in out}


def _exact_store(s):
    c = s["case"]
    cache = s["cache"].double()
    k = _turned(s, s["k"][:, None], c["R"])[:, 0]
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            cache[slot // c["P"], slot % c["P"], :c["C"]] = s["latent"][t].double()
            cache[slot // c["P"], slot % c["P"], c["C"]:] = k[t]
    return {"cache": cache, "q": _turned(s, s["q"], c["R"])}


def _exact_absorbed(s):
    c = s["case"]
    P, C = c["P"], c["C"]
    lens = s["lens"].tolist()
    cu = s["cu_q"].tolist() if s["cu_q"] is not None else list(range(c["B"] + 1))
    o = torch.zeros((*s["q"].shape[:2], C), dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        pages = s["table"][b, :_pages(lens[b], P)].long()
        kv = s["cache"][pages].double().flatten(0, 1)[:lens[b]]
        for i in range(cu[b], cu[b + 1]):
            seen = kv[:lens[b] - (cu[b + 1] - 1 - i)]
            x = s["q"][i].double() @ seen.T * s["scale"]
            o[i] = torch.softmax(x, dim=-1) @ seen[:, :C]
            lse[i] = torch.logsumexp(x, dim=-1)
    return {"out": o, "lse": lse}


def _exact_expanded(s):
    c = s["case"]
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    o = torch.zeros((*s["q"].shape[:2], c["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, L = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        unseen = torch.ones(n, L, dtype=torch.bool, device="cuda").triu(L - n + 1)
        for h in range(c["H"]):
            q, k = s["q"][rows, h].double(), s["k"][keys, h].double()
            x = (q[:, :c["Dn"]] @ k.T + q[:, c["Dn"]:] @ s["k_shared"][keys].double().T) * s["scale"]
            x = x.masked_fill(unseen, -math.inf)
            o[rows, h] = torch.softmax(x, dim=-1) @ s["v"][keys, h].double()
            lse[rows, h] = torch.logsumexp(x, dim=-1)
    return {"out": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return {n: _turned(s, s[n], case["rot"], case["back"]) for n in ("q", "k")}
    return {"append": _exact_append, "store": _exact_store, "absorbed": _exact_absorbed,
            "expanded": _exact_expanded}[case["op"]](s)
