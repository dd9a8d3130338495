"""A check of paged attention whose tolerance is each row's own.

tests/paged_ref.py bounds what fp16 weights lose below their normal range by the largest value scale
of the whole cache; here it is bounded by the largest contribution of the keys that the row sees, so that rows
of small values are held to their own size."""
import math

import numpy as np
import torch


def attend(cache, q, table, lens, cu, scale, causal, selected=None):
    """Per row of q [T, Hq, d] float64, from the definition: O, LSE, A = sum_j p_j |v_j| per channel,
    D = max_j scale sum_c |q_c k_jc|, C = max_j p_j s_j with s_j the scale of key j's value, n keys seen."""
    T, Hq, d = q.shape
    G, P = Hq // cache.Hk, cache.P
    O, A = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    L = np.full((T, Hq), -math.inf)
    D, C, N = np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n, length = int(cu[b + 1] - cu[b]), int(lens[b])
        if length == 0 or n == 0:
            continue
        k, v = cache.request(table[b], length, "k"), cache.request(table[b], length, "v")
        s = np.repeat(cache.scale["v"][table[b][:-(-length // P)]], P, axis=0)[:length]      # [length, Hk]
        rows = slice(int(cu[b]), int(cu[b + 1]))
        last = np.arange(n) + length - n if causal else np.full(n, length - 1)
        see = np.arange(length)[None, :] <= last[:, None]
        for h in range(Hq):
            kk, vv, qq, seen = k[h // G], v[h // G], q[rows, h], see
            if selected is not None:
                seen = see & np.isin(np.arange(length) // P, selected[b][h // G])[None, :]
            any_ = seen.any(axis=1)
            x = np.where(seen, scale * (qq @ kk.T), -math.inf)
            m = np.where(any_, x.max(axis=1), 0.0)
            p = np.exp(x - m[:, None])
            l = np.where(any_, p.sum(axis=1), 1.0)
            p /= l[:, None]
            O[rows, h], A[rows, h] = p @ vv, p @ np.abs(vv)
            L[rows, h] = np.where(any_, m + np.log(l), -math.inf)
            D[rows, h] = np.where(seen, scale * (np.abs(qq) @ np.abs(kk).T), 0.0).max(axis=1)
            C[rows, h] = (p * s[None, :, h // G]).max(axis=1)
            N[rows, h] = seen.sum(axis=1)
    return O, L, A, D, C, N


def tolerances(got, d, dtype, log2_top=6):
    """What the kernels' arithmetic may be off by, row by row.
    Scores: exact products, d additions in fp32 (each off by at most 2^-23 of the sum of sizes) and two fp32
    operations: (d + 4) 2^-23 D.  Base-2 exponents of at most 2^log2_top in size: three more roundings
    of half a step, 3 * 2^(log2_top - 24) * ln 2, and 2^-22 of 2^x itself: together delta, with 2^(log2_top - 23)
    for the last two (2^-22 is below a quarter of it).
    LSE: delta, n 2^-24 from the sum, 2^-22 |LSE|.
    O: weights off by delta each, in the sum above and the one below (2 delta A), rounded to fp16 (half a step,
    2^-11 A), sums in fp32 (n 2^-23 A); a weight below fp16's normal range is off by at most 2^-25 where the row's
    largest contribution has a weight of at least 2^8, and a code is at most 448: n 2^-33 448 C.
    Then the output's rounding, half a step: eps / 2, or half the type's smallest number."""
    O, L, A, D, C, N = got
    delta = (d + 4) * 2.0 ** -23 * D + 2.0 ** (log2_top - 23)
    lse = delta + N * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0))
    o = (2 * delta + 2.0 ** -11 + N * 2.0 ** -23)[..., None] * A + (N * 2.0 ** -33 * 448 * C)[..., None]
    f = torch.finfo(dtype)
    return o + (np.abs(O) + o) * f.eps / 2 + f.smallest_normal * f.eps / 2, lse


def mismatch(o, l, got, d, dtype, log2_top=6):
    """What of the outputs o [T, Hq, d] and l [T, Hq] (float64) is wrong: texts, empty where nothing is."""
    O, L = got[:2]
    to, tl = tolerances(got, d, dtype, log2_top)
    empty, wrong = ~np.isfinite(L), []
    if not np.array_equal(l == -math.inf, empty) or not (o[empty] == 0).all():
        wrong.append("rows that see no key")
    if not np.isfinite(o).all() or not np.isfinite(l[~empty]).all():
        wrong.append("not finite")
        return wrong
    off = np.abs(l[~empty] - L[~empty]) / tl[~empty]
    if off.size and off.max() > 1:
        wrong.append(f"LSE off by {off.max():.3g} tolerances")
    off = np.abs(o - O) / to
    if off.max() > 1:
        wrong.append(f"O off by {off.max():.3g} tolerances")
    return wrong


def check(out, lse, got, d, dtype, log2_top=6):
    wrong = mismatch(out.double().cpu().numpy(), lse.double().cpu().numpy(), got, d, dtype, log2_top)
    assert not wrong, wrong


def blind(got, d, dtype, log2_top=6, part=0.1):
    """Of each (row, head) that sees a key, the part of its channels whose tolerance passes `part` of the row's
    root-mean-square output: where it is 1 any small output would pass."""
    O, L = got[:2]
    to, _ = tolerances(got, d, dtype, log2_top)
    size = np.sqrt((O ** 2).mean(axis=-1, keepdims=True))
    return (to > part * size).mean(axis=-1)[np.isfinite(L)]
