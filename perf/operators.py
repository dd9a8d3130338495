"""Cases of the serving operators around a paged key/value cache held in 8 bits, in plain
torch operations and as the framework's calls.

The cache: pages of `P` tokens; k and v [pages, Hk, P, d] in e4m3, with one power-of-two
scale per page and key head ([pages, Hk], fp32): a value is code * scale.  A request owns
the pages its row of the block table lists; its token j lies in page table[j // P], place
j % P.  Four operators:

  tables  one serving step's bookkeeping: requests release their pages or take new ones
          from a stack of free pages, and every new token gets its slot (page * P + place)
  append  new keys and values quantised into their slots; a page's scale grows when a
          larger value arrives (its older codes are then rounded again to the new scale)
  attend  attention of each request's new queries over its cached keys (bottom-right
          causal mask, grouped heads), with the log-sum-exp
  sparse  for one query per request: an integer score of every page from the bounds of its
          keys, the best pages of each key head, and attention over those pages alone
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
        # a decode step of a small batch: every request adds one token, a few need a page
        {"name": "tables, small decode step", "op": "tables", "B": 8, "P": 64, "len": 4096,
         "new": 1, "ends": 0.0, "prompts": 0.0},
        # a busy server's step: most requests add a token, some end, some bring a prompt
        {"name": "tables, mixed step", "op": "tables", "B": 1000, "P": 16, "len": 2000,
         "new": 1, "ends": 0.06, "prompts": 0.04},
        # a batch of prompts enters at once
        {"name": "tables, prompts", "op": "tables", "B": 128, "P": 64, "len": 0, "new": 4000,
         "ends": 0.0, "prompts": 0.0},
        # the tokens of one decode step
        {"name": "append, decode step", "op": "append", "B": 32, "Hk": 8, "d": 128, "P": 64,
         "len": 4096, "new": 1, "dtype": "bf16", "bounds": True},
        # odd head count and width, short ragged pieces of prompts that start inside pages
        {"name": "append, ragged pieces", "op": "append", "B": 20, "Hk": 5, "d": 96, "P": 32,
         "len": 333, "new": 150, "dtype": "fp16", "bounds": True},
        # whole prompts written at once
        {"name": "append, prompts", "op": "append", "B": 8, "Hk": 8, "d": 128, "P": 64, "len": 0,
         "new": 8192, "dtype": "bf16", "bounds": False},
        # one user's next token after a context of 4096
        {"name": "attend, one request", "op": "attend", "B": 1, "Hq": 32, "Hk": 8, "d": 128,
         "P": 64, "len": 4096, "new": 1, "dtype": "bf16"},
        # the next tokens of a ragged batch with contexts up to 16384
        {"name": "attend, ragged batch", "op": "attend", "B": 64, "Hq": 32, "Hk": 8, "d": 128,
         "P": 64, "len": 16384, "new": 1, "dtype": "bf16"},
        # wide heads and small pages
        {"name": "attend, wide heads", "op": "attend", "B": 16, "Hq": 16, "Hk": 2, "d": 256,
         "P": 16, "len": 8192, "new": 1, "dtype": "fp16"},
        # pieces of long prompts read against what is cached already
        {"name": "attend, prompt pieces", "op": "attend", "B": 3, "Hq": 32, "Hk": 8, "d": 128,
         "P": 64, "len": 8192, "new": 2048, "dtype": "bf16"},
        # one user's next token after a long context, 64 pages read
        {"name": "sparse, one request", "op": "sparse", "B": 1, "Hq": 32, "Hk": 8, "d": 128,
         "P": 16, "len": 16384, "keep": 64, "dtype": "bf16"},
        # a ragged batch with long contexts, 64 pages read
        {"name": "sparse, ragged batch", "op": "sparse", "B": 32, "Hq": 32, "Hk": 8, "d": 128,
         "P": 64, "len": 32768, "keep": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "sparse"])
    P = rng.choice([16, 32, 64, 128])
    if op == "tables":
        if rng.random() < 0.5:
            return {"op": op, "B": _log(rng, 1, 1500), "P": P, "len": _log(rng, 1, 4000), "new": 1,
                    "ends": rng.choice([0.0, 0.05, 0.3]), "prompts": rng.choice([0.0, 0.05])}
        return {"op": op, "B": _log(rng, 1, 128), "P": P, "len": rng.choice([0, 100]),
                "new": _log(rng, 2, 3900), "ends": 0.0, "prompts": 0.0}
    Hk, d = rng.choice([1, 2, 3, 5, 8]), rng.choice([64, 80, 96, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        one = rng.random() < 0.4
        return {"op": op, "B": _log(rng, 1, 256) if one else _log(rng, 1, 8), "Hk": Hk, "d": d, "P": P,
                "len": _log(rng, 1, 2000) if one else rng.choice([0, _log(rng, 1, 500)]),
                "new": 1 if one else _log(rng, 2, 4000), "dtype": dtype, "bounds": rng.random() < 0.5}
    G = rng.choice([1, 2, 3, 4, 5, 8])
    c = {"op": op, "B": _log(rng, 1, 32), "Hq": Hk * G, "Hk": Hk, "d": d, "P": P,
         "len": _log(rng, 1, 12000), "dtype": dtype}
    if op == "sparse":
        c["keep"] = _log(rng, 2, 100)
        return c
    kind = rng.random()
    if kind < 0.5:
        c["new"] = 1
    elif kind < 0.75:  # a few tokens at once: drafts that are checked together
        c["new"] = rng.randint(2, 16)
    else:
        c["B"], c["len"], c["new"] = rng.randint(1, 3), _log(rng, 100, 6000), _log(rng, 17, 2000)
    return c


def _spread(n, top, low):
    """n whole numbers in [low * top, top], ragged, the first one `top`."""
    f = (np.arange(n) * 0.6180339887498949) % 1.0
    return np.maximum(1, np.floor(top * (1.0 - (1.0 - low) * f))).astype(np.int64)


def _sizes(c):
    """(tokens cached before the step, new tokens; negative: the request ends) of each request."""
    B = c["B"]
    lens = _spread(B, c["len"], 0.3) if c["len"] else np.zeros(B, np.int64)
    new = _spread(B, c.get("new", 1), 0.4)
    if c["op"] == "tables":
        u = (np.arange(B) * 0.7548776662466927 + 0.5) % 1.0
        new = np.where(u < c["ends"], -1, np.where(u > 1.0 - c["prompts"], 1 + (lens * 3) // 4, new))
    elif c["op"] == "attend":  # "len" counts the new tokens too
        new = np.minimum(new, lens)
        lens = lens - new
    elif c["op"] == "sparse":
        lens = lens - 1
    return lens, new


def _pages(n, P):
    return -(-n // P)


# --------------------------------------------------------------- inputs
def _scale_of(amax):
    """Smallest power of two s in [2^-60, 2^60] with amax <= 448 s (s = 2^60 where none is)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), e)


def _round_e4m3(x):
    return x.clamp(-_E4M3_MAX, _E4M3_MAX).to(_E4M3)  # NaN stays NaN


def _random_cache(g, pages, Hk, P, d):
    """Codes and scales of pages of keys or values whose size differs by page and head."""
    codes = torch.empty((pages, Hk, P, d), dtype=_E4M3, device="cuda")
    scales = torch.empty((pages, Hk), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (Hk * P * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((n, Hk, P, d), device="cuda", generator=g)
        x *= torch.exp(0.4 * torch.randn((n, Hk, 1, 1), device="cuda", generator=g))
        s = _scale_of(x.abs().amax(dim=(2, 3)))
        codes[i:i + n] = _round_e4m3(x / s[:, :, None, None])
        scales[i:i + n] = s
    return codes, scales


def _bounds_of(codes, filled):
    """Per page, head and channel: floor and ceil of (least, largest code) / 4 over the filled
    places, as [pages, Hk, 2, d] int8."""
    x = codes.float().nan_to_num(nan=0.0)
    at = torch.arange(x.shape[2], device=x.device)[None, :] < filled[:, None]
    at = at[:, None, :, None]
    lo = torch.where(at, x, torch.full_like(x, math.inf)).amin(dim=2)
    hi = torch.where(at, x, torch.full_like(x, -math.inf)).amax(dim=2)
    return torch.stack([torch.floor(lo / 4), torch.ceil(hi / 4)], dim=2).to(torch.int8)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    P, B = c["P"], c["B"]
    before, new = _sizes(c)
    after = np.where(new < 0, 0, before + np.maximum(new, 0))
    held = _pages(np.maximum(before, after), P) if c["op"] != "append" else _pages(after, P)
    if c["op"] == "tables":
        have = _pages(before, P)
        need = np.where(new < 0, 0, _pages(after, P) - have)
        M = int(max(have.max(), _pages(after, P).max())) + 3
        spare = 5
        pool = int(have.sum() + need.sum()) + spare
        perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
        table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(M, device="cuda")[None, :] < torch.as_tensor(have, device="cuda")[:, None]
        table[col] = perm[:int(have.sum())]
        free = torch.zeros(pool, dtype=torch.int32, device="cuda")
        nfree = pool - int(have.sum())
        free[:nfree] = perm[int(have.sum()):]
        tokens = int(np.maximum(new, 0).sum())
        return {"case": c, "new": _i32(new), "lens": _i32(before), "table": table, "free": free,
                "count": _i32([nfree]), "tokens": tokens + 3}
    Hk, d = c["Hk"], c["d"]
    pool, M = int(held.sum()) + 7, int(held.max())
    table = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    col = torch.arange(M, device="cuda")[None, :] < torch.as_tensor(held, device="cuda")[:, None]
    table[col] = torch.randperm(pool, device="cuda", generator=g)[:int(held.sum())].to(torch.int32)
    s = {"case": c, "table": table, "lens": _i32(after)}
    dt = _TYPES[c["dtype"]]
    s["k_cache"], s["k_scale"] = _random_cache(g, pool, Hk, P, d)
    s["v_cache"], s["v_scale"] = _random_cache(g, pool, Hk, P, d)
    if c["op"] == "append":
        T = int(new.sum())
        req = np.repeat(np.arange(B), new)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(before, new)])
        req_t, pos_t = torch.as_tensor(req, device="cuda"), torch.as_tensor(pos, device="cuda")
        slots = table[req_t, pos_t // P].long() * P + pos_t % P
        # two padding rows at the end, as a step of fixed size has them
        s["slots"] = torch.cat([slots, torch.full((2,), -1, device="cuda")]).to(torch.int32)
        # projections come as one [T, 2, Hk, d] tensor: k and v are views of it
        kv = torch.randn((T + 2, 2, Hk, d), device="cuda", generator=g)
        kv *= torch.exp(0.4 * torch.randn((T + 2, 2, Hk, 1), device="cuda", generator=g))
        kv = kv.to(dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["bounds"] = None
        if c["bounds"]:
            filled = torch.zeros(pool, dtype=torch.int64, device="cuda")
            j = torch.arange(M, device="cuda")[None, :]
            b4 = torch.as_tensor(before, device="cuda")[:, None]
            filled[table[col].long()] = (b4 - j * P).clamp(0, P)[col]
            s["bounds"] = _bounds_of(s["k_cache"], filled.clamp(min=1))
        return s
    T = int(new.sum()) if c["op"] == "attend" else B
    s["q"] = torch.randn((T, c["Hq"], d), device="cuda", generator=g).to(dt)
    s["scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "attend":
        s["cu"] = _i32(np.concatenate([[0], np.cumsum(new)])) if c["new"] > 1 else None
        s["max_q"] = int(new.max())
    else:
        filled = torch.full((pool,), P, dtype=torch.int64, device="cuda")
        last = torch.as_tensor(held - 1, device="cuda")[:, None]
        filled[table.gather(1, last)[:, 0].long()] = torch.as_tensor(after - (held - 1) * P, device="cuda")
        s["bounds"] = torch.cat([_bounds_of(s["k_cache"][i:i + 512], filled[i:i + 512])
                                 for i in range(0, pool, 512)])
    return s


# --------------------------------------------------------- the plain forms
def _plain_tables(s):
    P, new, lens, table, free, count = s["case"]["P"], s["new"].long(), s["lens"].long(), s["table"], s["free"], s["count"].long()
    B, M = table.shape
    ends = new < 0
    add = new.clamp(min=0)
    after = torch.where(ends, 0, lens + add)
    have = (lens + P - 1) // P
    need = torch.where(ends, 0, (after + P - 1) // P - have)
    back = torch.where(ends, have, 0)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    good = (need.sum() <= count[0] + back.sum()) & (cu[-1] <= s["tokens"]) & (have.maximum((after + P - 1) // P).max() <= M) \
        & (count[0] + back.sum() <= free.numel())
    j = torch.arange(M, device=new.device)[None, :]
    # pages of ended requests go back on top of the stack, in order
    to = count + (back.cumsum(0) - back)[:, None] + j
    to = torch.where((j < back[:, None]) & good, to, free.numel())
    pile = torch.cat([free, free.new_zeros(1)]).scatter(0, to.reshape(-1), table.reshape(-1))[:-1]
    # new pages come off the top, in order
    top = count[0] + back.sum()
    nth = (need.cumsum(0) - need)[:, None] + j - have[:, None]
    take = (j >= have[:, None]) & (j < (have + need)[:, None]) & good
    out = torch.where(take, pile[(top - 1 - nth).clamp(0, free.numel() - 1)], table)
    t = torch.arange(s["tokens"], device=new.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, B - 1)
    pos = lens[b] + t - cu[b]
    slots = out[b, (pos // P).clamp(0, M - 1)].long() * P + pos % P
    slots = torch.where((t < cu[-1]) & good, slots, -1)
    return {"slots": slots.int(), "cu": torch.where(good, cu, 0).int(), "lens": torch.where(good, after, lens).int(),
            "count": torch.where(good, top - need.sum(), count).int(), "table": out, "free": pile}


def _plain_append(s):
    c = s["case"]
    P, slots = c["P"], s["slots"].long()
    keep = slots >= 0
    slots = slots[keep]
    pages, at = torch.unique(slots // P, return_inverse=True)
    place = slots % P
    n, Hk, d = pages.numel(), c["Hk"], c["d"]
    first = torch.full((n,), P, device=slots.device).scatter_reduce(0, at, place, "amin")
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[keep].float()
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
    if s["bounds"] is not None:
        filled = torch.zeros(n, dtype=torch.int64, device=slots.device).scatter_reduce(0, at, place + 1, "amax")
        s["bounds"][pages] = _bounds_of(s["k_cache"][pages], filled)
    out = {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out if s["bounds"] is None else dict(out, bounds=s["bounds"])


def _softmax_sum(x, v):
    """(weighted mean of v, log-sum-exp) over the last axis of scores x; rows that see nothing: 0, -inf."""
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    B, Hk, P, d, G = c["B"], c["Hk"], c["P"], c["d"], c["Hq"] // c["Hk"]
    table, lens = s["table"].long(), s["lens"].long()
    M, n = table.shape[1], s["max_q"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=lens.device)
    i = torch.arange(n, device=lens.device)
    have = i[None, :] < (cu[1:] - cu[:-1])[:, None]                       # [B, n]
    row = torch.where(have, cu[:-1, None] + i, 0)
    q = s["q"].float()[row].view(B, n, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, d)

    def whole(cache, scale):
        x = cache[table].float() * scale[table][:, :, :, None, None]      # [B, M, Hk, P, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, M * P, d)

    x = torch.matmul(q, whole(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    j = torch.arange(M * P, device=lens.device)
    last = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + i                # [B, n]
    see = (j[None, None, :] < lens[:, None, None]) & (j[None, None, :] <= last[:, :, None])
    x = x.view(B, Hk, G, n, M * P).masked_fill_(~see[:, None, None], -math.inf).view(B, Hk, G * n, M * P)
    o, lse = _softmax_sum(x, whole(s["v_cache"], s["v_scale"]))
    o = o.view(B, Hk, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hk * G, d)[have]
    lse = lse.view(B, Hk, G, n).permute(0, 3, 1, 2).reshape(B, n, Hk * G)[have]
    return {"out": o.to(s["q"].dtype), "lse": lse}


def _plain_sparse(s):
    c = s["case"]
    B, Hk, P, d, G, keep = c["B"], c["Hk"], c["P"], c["d"], c["Hq"] // c["Hk"], c["keep"]
    table, lens = s["table"].long(), s["lens"].long()
    M = table.shape[1]
    q = s["q"].float()
    # whole-number queries: the smallest power of two u with |q| <= 127 u, then q / u rounded
    a = q.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(a)
    e = torch.where(m <= 127 / 128, e - 7, e - 6)
    u = torch.ldexp(torch.ones_like(a), torch.where(a > 0, e, torch.full_like(e, -60)).clamp(-60, 60))
    qi = torch.round(q / u).clamp(-127, 127).view(B, Hk, G, d)
    b = s["bounds"][table].permute(0, 2, 3, 4, 1).float()                 # [B, Hk, 2, d, M]
    # products of whole numbers: sums below 2^24, so exact in 32 bits
    x = torch.matmul(qi.clamp(max=0), b[:, :, 0]) + torch.matmul(qi.clamp(min=0), b[:, :, 1])
    x = x * (u.view(B, Hk, G, 1) * (4.0 * s["k_scale"][table].permute(0, 2, 1))[:, :, None])
    x = x.amax(dim=2)                                                     # [B, Hk, M]
    pages = ((lens + P - 1) // P)[:, None, None]
    j = torch.arange(M, device=lens.device)
    x = torch.where(j == pages - 1, math.inf, torch.where(j < pages, x, -math.inf))
    best = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :, :keep]
    if M < keep:
        best = torch.cat([best, torch.full((B, Hk, keep - M), M, device=lens.device)], dim=-1)
    best = torch.where(best < pages, best, M).sort(dim=-1)[0]
    sel = torch.where(best < M, best, -1)
    count = (sel >= 0).sum(dim=-1)
    # attention over the kept pages
    page = table[:, None, :].expand(B, Hk, M).gather(2, sel.clamp(min=0))  # [B, Hk, keep]
    head = torch.arange(Hk, device=lens.device)[None, :, None]

    def some(cache, scale):
        return (cache.view(torch.uint8)[page, head].view(_E4M3).float() * scale[page, head][..., None, None]).view(B, Hk, keep * P, d)

    x = torch.matmul(q.view(B, Hk, G, d), some(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    pos = (sel[..., None] * P + torch.arange(P, device=lens.device)).view(B, Hk, 1, keep * P)
    see = (sel >= 0)[..., None].expand(B, Hk, keep, P).reshape(B, Hk, 1, keep * P) & (pos < lens[:, None, None, None])
    o, lse = _softmax_sum(x.masked_fill(~see, -math.inf), some(s["v_cache"], s["v_scale"]))
    return {"selected": sel.int(), "count": count.int(), "out": o.view(B, Hk * G, d).to(s["q"].dtype), "lse": lse.view(B, Hk * G)}


def _own(s):
    import online_softmax_tiling_gb300 as fa
    c = s["case"]
    if c["op"] == "tables":
        slots, cu, lens, count, _ = fa.kv_tables_step(s["new"], s["lens"], s["table"], s["free"], s["count"],
                                                      page_size=c["P"], max_tokens=s["tokens"])
        return {"slots": slots, "cu": cu, "lens": lens, "count": count, "table": s["table"], "free": s["free"]}
    if c["op"] == "append":
        fa.kv_cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                           k_bounds=s["bounds"])
        out = {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        return out if s["bounds"] is None else dict(out, bounds=s["bounds"])
    if c["op"] == "attend":
        o, lse = fa.paged_attention_forward(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                            s["table"], s["lens"], cu_q=s["cu"], max_q=s["max_q"],
                                            scale=s["scale"], causal=True)
        return {"out": o, "lse": lse}
    sel, count = fa.kv_page_select(s["q"], s["bounds"], s["k_scale"], s["table"], s["lens"],
                                   page_size=c["P"], num_selected=c["keep"])
    o, lse = fa.paged_attention_forward(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                        s["table"], s["lens"], scale=s["scale"], selected=sel,
                                        selected_count=count)
    return {"selected": sel, "count": count, "out": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend,
            "sparse": _plain_sparse}[state["case"]["op"]](state)


def work(case):
    c = case
    P, B = c["P"], c["B"]
    before, new = _sizes(c)
    if c["op"] == "tables":
        tokens = int(np.maximum(new, 0).sum()) + 3
        have = _pages(before, P)
        moved = int(np.where(new < 0, have, _pages(before + np.maximum(new, 0), P) - have).sum())
        # lengths and counts in and out, each moved page read and written, the page of every
        # page of tokens read, every slot written
        return {"bytes": 4.0 * (4 * B + 2 * moved + tokens + tokens / P), "flops": 0.0}
    Hk, d = c["Hk"], c["d"]
    if c["op"] == "append":
        T = int(new.sum())
        pages = int((_pages(before + new, P) - before // P).sum())
        b = T * Hk * d * 2 * 2 + T * Hk * d * 2 + 4 * (T + 2) + pages * Hk * 2 * 8
        if c["bounds"]:
            b += pages * Hk * 2 * d + int((before % P > 0).sum()) * Hk * 2 * d
        return {"bytes": float(b), "flops": 3.0 * T * Hk * d * 2}
    Hq, after = c["Hq"], before + new
    if c["op"] == "attend":
        # pairs of a query and a key it sees
        pairs = float((new * before + new * (new + 1) // 2).sum())
        keys, T = float(after.sum()), int(new.sum())
        b = keys * Hk * d * 2 + _pages(after, P).sum() * (4 + Hk * 8) + T * Hq * (d * 4 + 4)
        return {"bytes": float(b), "flops": 4.0 * pairs * Hq * d}
    pages = _pages(after, P)
    kept = np.minimum(pages, c["keep"])
    keys = float(np.where(pages <= c["keep"], after, (kept - 1) * P + after - (pages - 1) * P).sum())
    b = float(pages.sum()) * (Hk * (2 * d + 4) + 4) + keys * Hk * d * 2 + float(kept.sum()) * Hk * (8 + 4) \
        + B * Hq * (d * 4 + 4)
    return {"bytes": b, "flops": 4.0 * keys * Hq * d + 2.0 * float(pages.sum()) * Hq * d}


# ----------------------------------------- the definitions, in 64 bits or whole numbers
def _exact_tables(s):
    P = s["case"]["P"]
    new, lens, table = (s[k].cpu().numpy().astype(np.int64) for k in ("new", "lens", "table"))
    free, top = s["free"].cpu().numpy().astype(np.int64).copy(), int(s["count"][0])
    table, slots, cu, after = table.copy(), np.full(s["tokens"], -1), [0], []
    for b, n in enumerate(new):
        if n < 0:
            for j in range(-(-lens[b] // P)):
                free[top] = table[b, j]
                top += 1
    pile = free.copy()
    for b, n in enumerate(new):
        if n < 0:
            after.append(0)
            cu.append(cu[-1])
            continue
        for j in range(-(-lens[b] // P), -(-(lens[b] + n) // P)):
            top -= 1
            table[b, j] = pile[top]
        pos = np.arange(lens[b], lens[b] + n)
        slots[cu[-1]:cu[-1] + n] = table[b, pos // P] * P + pos % P
        cu.append(cu[-1] + n)
        after.append(lens[b] + n)
    return {"slots": slots.astype(np.int32), "cu": np.array(cu, np.int32), "lens": np.array(after, np.int32),
            "count": np.array([top], np.int32), "table": table.astype(np.int32), "free": pile.astype(np.int32)}


def _nearest_e4m3(x):
    """float64 -> the nearest e4m3 number (ties to even), at most 448 in size, as float64."""
    with np.errstate(invalid="ignore"):
        e = np.maximum(np.frexp(x)[1] - 1, -6)
        q = np.ldexp(1.0, e - 3)
        return np.clip(np.where(np.isinf(x), x, np.rint(x / q) * q), -448.0, 448.0)


def _exact_append(s):
    P = s["case"]["P"]
    slots = s["slots"].cpu().numpy()
    runs, t = [], 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] // P == slots[t] // P:
            n += 1
        runs.append((t, n, slots[t] // P, slots[t] % P))
        t += n
    out = {}
    for name in ("k", "v"):
        x = s[name].double().cpu().numpy()
        codes = s[name + "_cache"].float().cpu().numpy()
        scales = s[name + "_scale"].cpu().numpy().astype(np.float64)
        for t, n, page, place in runs:
            y = x[t:t + n].transpose(1, 0, 2)                             # [Hk, n, d]
            top = np.abs(y).max(axis=(1, 2))
            want = np.exp2(np.clip(np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -60, 60))
            want = np.where(top > want * 448.0, want * 2, want)
            want = np.where(top <= want * 224.0, want / 2, want)
            now = want if place == 0 else np.maximum(want, scales[page])
            if place and (now > scales[page]).any():
                codes[page, :, :place] = _nearest_e4m3(codes[page, :, :place] * (scales[page] / now)[:, None, None])
            codes[page, :, place:place + n] = _nearest_e4m3(y / now[:, None, None])
            scales[page] = now
        out[name], out[name + "_scale"] = codes.astype(np.float32), scales.astype(np.float32)
    if s["bounds"] is not None:
        bounds = s["bounds"].cpu().numpy().copy()
        for t, n, page, place in runs:
            z = out["k"][page, :, :place + n]
            bounds[page, :, 0], bounds[page, :, 1] = np.floor(z.min(axis=1) / 4), np.ceil(z.max(axis=1) / 4)
        out["bounds"] = bounds
    return out


def _request(s, b, pages, head=None):
    """Keys and values of the given pages of request b in 64 bits: [Hk or 1, keys, d] each."""
    idx = s["table"][b, pages].long()
    got = []
    for name in ("k", "v"):
        x, f = s[name + "_cache"].view(torch.uint8)[idx], s[name + "_scale"][idx].double()
        if head is not None:
            x, f = x[:, head:head + 1], f[:, head:head + 1]
        x = x.contiguous().view(_E4M3).double() * f[:, :, None, None]
        got.append(x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3]))
    return got


def _exact_attend(s):
    c = s["case"]
    G, P = c["Hq"] // c["Hk"], c["P"]
    lens = s["lens"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(c["B"] + 1))
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n, L = cu[b + 1] - cu[b], lens[b]
        k, v = _request(s, b, slice(0, _pages(L, P)))
        for h in range(c["Hq"]):
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k[h // G, :L].T * s["scale"]
            x = x.masked_fill(torch.ones(n, L, dtype=torch.bool, device="cuda").triu(L - n + 1), -math.inf)
            o[cu[b]:cu[b + 1], h] = torch.softmax(x, dim=-1) @ v[h // G, :L]
            lse[cu[b]:cu[b + 1], h] = torch.logsumexp(x, dim=-1)
    return {"out": o, "lse": lse}


def _exact_sparse(s):
    c = s["case"]
    Hk, G, P, keep = c["Hk"], c["Hq"] // c["Hk"], c["P"], c["keep"]
    bounds, ks = s["bounds"].cpu().numpy().astype(np.int64), s["k_scale"].cpu().numpy().astype(np.float64)
    table, lens, q = s["table"].cpu().numpy(), s["lens"].tolist(), s["q"].double().cpu().numpy()
    sel = np.full((c["B"], Hk, keep), -1, np.int32)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n = _pages(lens[b], P)
        for h in range(Hk):
            score = np.full(n, -np.inf)
            for g in range(G):
                y = q[b, h * G + g]
                u = -60
                while np.abs(y).max() > 127.0 * 2.0 ** u:
                    u += 1
                z = np.rint(y / 2.0 ** u).astype(np.int64)
                lo, hi = bounds[table[b, :n], h, 0], bounds[table[b, :n], h, 1]
                score = np.maximum(score, np.maximum(lo * z, hi * z).sum(axis=1) * 2.0 ** u * 4.0 * ks[table[b, :n], h])
            score[n - 1] = np.inf
            pick = np.sort(np.lexsort((np.arange(n), -score))[:keep])
            sel[b, h, :len(pick)] = pick
            pages = torch.as_tensor(pick, device="cuda")
            k, v = _request(s, b, pages, h)
            pos = (pages[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
            x = s["q"][b, h * G:(h + 1) * G].double() @ k[0].T * s["scale"]
            x = x.masked_fill(pos >= lens[b], -math.inf)
            o[b, h * G:(h + 1) * G] = torch.softmax(x, dim=-1) @ v[0]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1)
    return {"selected": sel, "count": (sel >= 0).sum(axis=2).astype(np.int32), "out": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "attend": _exact_attend,
            "sparse": _exact_sparse}[case["op"]](s)
