"""The paged-cache operators from their definitions, in 64 bits or whole numbers on the CPU,
and random caches.  No code of the package is used."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def e4m3_values():
    """The 256 codes' values (S.1111.111 is NaN), from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (e == 15 and m == 7) else (-v if s else v)
    return out


VALUES = e4m3_values()


def round_e4m3(x):
    """float64 array -> codes (uint8): nearest, ties to the even code, at most 448, NaN kept."""
    pos = VALUES[:127]                                    # ascending, 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, np.nan_to_num(a)), 1, 126)
    lo = hi - 1
    below = a - pos[lo]
    above = pos[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def scale_of(x):
    """Smallest power of two s in [2^-60, 2^60] with |x| <= 448 s for every finite x."""
    a = np.abs(x[np.isfinite(x)])
    top = a.max() if a.size else 0.0
    e = -60
    while e < 60 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """A cache on the CPU: codes uint8, scales float64, bounds int8."""

    def __init__(self, pages, Hk, P, d, seed=0, random=True):
        rng = np.random.default_rng(seed)
        self.P, self.d, self.Hk, self.pages = P, d, Hk, pages
        self.codes, self.scale = {}, {}
        for n in "kv":
            if random:
                x = rng.standard_normal((pages, Hk, P, d)) * np.exp(0.5 * rng.standard_normal((pages, Hk, 1, 1)))
                s = 2.0 ** np.ceil(np.log2(np.abs(x).max(axis=(2, 3)) / 448.0))
                self.codes[n] = round_e4m3(x / s[:, :, None, None])
                self.scale[n] = s
            else:
                self.codes[n] = np.zeros((pages, Hk, P, d), np.uint8)
                self.scale[n] = np.zeros((pages, Hk))
        self.bounds = np.zeros((pages, Hk, 2, d), np.int8)

    def set_bounds(self, page, filled):
        x = np.nan_to_num(VALUES[self.codes["k"][page][:, :filled]], nan=0.0)
        self.bounds[page, :, 0] = np.floor(x.min(axis=1) / 4)
        self.bounds[page, :, 1] = np.ceil(x.max(axis=1) / 4)

    def append(self, k, v, slots, bounds=True):
        """k, v [T, Hk, d] float64."""
        t = 0
        while t < len(slots):
            if slots[t] < 0:
                t += 1
                continue
            page, place, n = slots[t] // self.P, slots[t] % self.P, 1
            while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] // self.P == page:
                n += 1
            # bounds of what the page held: they stand unless the scale of its keys grows
            held, grew = self.bounds[page].astype(int), np.zeros(self.Hk, bool)
            for name, x in (("k", k), ("v", v)):
                for h in range(self.Hk):
                    s = scale_of(x[t:t + n, h])
                    old = self.scale[name][page, h]
                    c = self.codes[name][page, h]
                    if place:
                        s = max(s, old)
                        if s > old:
                            grew[h] |= name == "k"
                            c[:place] = round_e4m3(VALUES[c[:place]] * (old / s))
                    c[place:place + n] = round_e4m3(x[t:t + n, h] / s)
                    self.scale[name][page, h] = s
            if bounds:
                self.set_bounds(page, place + n)
                if place:
                    x = np.nan_to_num(VALUES[self.codes["k"][page][:, place:place + n]], nan=0.0)
                    lo = np.minimum(held[:, 0], np.floor(x.min(axis=1) / 4))
                    hi = np.maximum(held[:, 1], np.ceil(x.max(axis=1) / 4))
                    self.bounds[page, ~grew, 0], self.bounds[page, ~grew, 1] = lo[~grew], hi[~grew]
            t += n

    def cuda(self):
        """(k_cache, v_cache, k_scale, v_scale, k_bounds) on the GPU."""
        t = [torch.from_numpy(self.codes[n].copy()).cuda().view(E4M3) for n in "kv"]
        t += [torch.from_numpy(self.scale[n].astype(np.float32)).cuda() for n in "kv"]
        return (*t, torch.from_numpy(self.bounds.copy()).cuda())

    def request(self, row, length, name):
        """Values [Hk, length, d] of a request."""
        n = -(-length // self.P)
        x = VALUES[self.codes[name][row[:n]]] * self.scale[name][row[:n]][:, :, None, None]
        return x.transpose(1, 0, 2, 3).reshape(self.Hk, n * self.P, self.d)[:, :length]


def attend(cache, q, table, lens, cu, scale, causal, selected=None):
    """(O, LSE, A, D): q [T, Hq, d] float64; A = sum_j p_j |v_j| per channel, D = max_j scale sum_c |q_c k_jc|
    per row (for tolerances)."""
    T, Hq, d = q.shape
    G = Hq // cache.Hk
    O, A = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    L, D = np.full((T, Hq), -math.inf), np.zeros((T, Hq))
    for b in range(len(lens)):
        n, length = cu[b + 1] - cu[b], int(lens[b])
        if length == 0 or n == 0:
            continue
        k, v = cache.request(table[b], length, "k"), cache.request(table[b], length, "v")
        for h in range(Hq):
            for i in range(n):
                see = np.arange(length) <= (i + length - n if causal else length)
                if selected is not None:
                    see &= np.isin(np.arange(length) // cache.P, selected[b][h // G])
                if not see.any():
                    continue
                kk, vv, row = k[h // G][see], v[h // G][see], q[cu[b] + i, h]
                x = scale * (kk @ row)
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                t = cu[b] + i
                O[t, h], A[t, h] = p @ vv / l, p @ np.abs(vv) / l
                L[t, h], D[t, h] = m + math.log(l), scale * (np.abs(kk) @ np.abs(row)).max()
    return O, L, A, D


def tolerances(O, L, A, D, d, n_keys, v_top, dtype):
    """What the kernel's arithmetic may be off by.
    Scores: exact products, d additions in fp32 (each off by at most 2^-23 of the sum of sizes), then
    two fp32 operations: delta = (d + 4) 2^-23 D, plus the 2^-22 of 2^x and of the subtraction of
    maxima up to |x| = 2^6 (2^-17).  LSE: delta, n 2^-24 from the sum, 2^-22 |L|.
    O: weights off by delta each (2 delta A), rounded to fp16 (2^-11 A), or below its normal range
    by 2^-25 against a largest weight of at least 2^8 (n 2^-33 of the largest value), sums in fp32 (n 2^-23 A);
    then the output's rounding, half a step: eps / 2, or half the type's smallest number."""
    delta = (d + 4) * 2.0 ** -23 * D + 2.0 ** -17
    lse = delta + n_keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0))
    o = (2 * delta[..., None] + 2.0 ** -11 + n_keys * 2.0 ** -23) * A + n_keys * 2.0 ** -33 * v_top
    f = torch.finfo(dtype)
    return o + (np.abs(O) + o) * f.eps / 2 + f.smallest_normal * f.eps / 2, lse


def check(out, lse, ref, d, n_keys, v_top, dtype, rows=slice(None)):
    O, L, A, D = (x[rows] for x in ref)
    to, tl = tolerances(O, L, A, D, d, n_keys, v_top, dtype)
    o, l = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    empty = ~np.isfinite(L)
    assert np.array_equal(l == -math.inf, empty)
    assert np.isfinite(o).all() and (o[empty] == 0).all()
    off = np.abs(l[~empty] - L[~empty])
    assert (off <= tl[~empty]).all(), (off / tl[~empty]).max()
    assert (np.abs(o - O) <= to).all(), (np.abs(o - O) / to).max()


def page_scores(cache, q, row, length):
    """Scores [Hk, pages] of one query [Hq, d] float64."""
    n, G = -(-length // cache.P), q.shape[0] // cache.Hk
    out = np.full((cache.Hk, n), -math.inf)
    for h in range(q.shape[0]):
        a = np.abs(np.nan_to_num(q[h], nan=0.0)).max()
        e = -60
        while e < 60 and a > 127.0 * 2.0 ** e:
            e += 1
        z = np.clip(np.rint(np.nan_to_num(q[h], nan=0.0) / 2.0 ** e), -127, 127)
        b = cache.bounds[row[:n], h // G].astype(np.float64)
        s = np.maximum(b[:, 0] * z, b[:, 1] * z).sum(axis=1) * 2.0 ** e * 4 * cache.scale["k"][row[:n], h // G]
        out[h // G] = np.maximum(out[h // G], s)
    return out


def select(cache, q, table, lens, keep):
    """(selected [B, Hk, keep], count [B, Hk])."""
    B = len(lens)
    sel, count = np.full((B, cache.Hk, keep), -1, np.int32), np.zeros((B, cache.Hk), np.int32)
    for b in range(B):
        if lens[b] == 0:
            continue
        s = page_scores(cache, q[b], table[b], int(lens[b]))
        n = s.shape[1]
        s[:, n - 1] = math.inf
        for h in range(cache.Hk):
            pick = np.sort(np.argsort(-s[h], kind="stable")[:keep])
            sel[b, h, :len(pick)], count[b, h] = pick, len(pick)
    return sel, count


def tables_step(new, lens, table, free, count, P, max_tokens):
    """One step on numpy arrays: dict of results; table and free as after the step."""
    B, M = table.shape
    after = np.where(new < 0, 0, lens + np.maximum(new, 0))
    have, want = -(-lens // P), -(-after // P)
    back = np.where(new < 0, have, 0).sum()
    need = np.where(new < 0, 0, want - have).sum()
    tokens = np.maximum(new, 0).sum()
    bad = (lens < 0).any() or (have > M).any() or (want > M).any() or tokens > max_tokens \
        or count < 0 or count + back > len(free)
    status = 1 if bad else 6 if need > count + back else 0
    table, free = table.copy(), free.copy()
    slots, cu = np.full(max_tokens, -1), np.zeros(B + 1, np.int64)
    if status:
        return dict(status=status, slots=slots, cu=cu, lens=lens, count=count, table=table, free=free)
    top = count
    for b in np.flatnonzero(new < 0):
        free[top:top + have[b]] = table[b, :have[b]]
        top += have[b]
    for b in range(B):
        cu[b + 1] = cu[b] + max(new[b], 0)
        if new[b] < 0:
            continue
        for j in range(have[b], want[b]):
            top -= 1
            table[b, j] = free[top]
        pos = np.arange(lens[b], after[b])
        slots[cu[b]:cu[b + 1]] = table[b, pos // P] * P + pos % P
    return dict(status=0, slots=slots, cu=cu, lens=after, count=top, table=table, free=free)
