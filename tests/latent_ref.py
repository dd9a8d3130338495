"""Rotary positions and latent attention from their definitions, on the CPU.  No code of the package is used."""
import math

import numpy as np
import torch


def table(n, dim, base=10000.0, factor=1.0):
    """[n, dim] float32: cosines, then sines."""
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(dim // 2) / dim)
    return (np.concatenate([np.cos(a), np.sin(a)], axis=1) * factor).astype(np.float32)


def turn(x, positions, tab, interleaved, inverse=False, dtype=np.float32):
    """x [T, heads, d] turned in `dtype`; float32: every product and sum rounded, as the operators define it."""
    x, tab = x.astype(dtype), tab.astype(dtype)
    h, y = tab.shape[1] // 2, x.astype(dtype).copy()
    on = (positions >= 0) & (positions < len(tab))
    row = tab[np.where(on, positions, 0)][:, None]
    c, s = row[..., :h], row[..., h:]
    if inverse:
        s = -s
    i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return np.where(on[:, None, None], y, x)


def attend(q, keys, values, limits, scale):
    """Rows q [n, H, D] over keys [m, D] or [m, H, D] and values: (O, LSE, A, S), row i seeing the first limits[i]
    keys; A = sum_j p_j |v_j|, S = max_j scale sum_c |q_c k_jc| (for tolerances)."""
    n, H, _ = q.shape
    dv = values.shape[-1]
    O, A = np.zeros((n, H, dv)), np.zeros((n, H, dv))
    L, S = np.full((n, H), -math.inf), np.zeros((n, H))
    for i in range(n):
        m = int(limits[i])
        if m <= 0:
            continue
        k = keys[:m] if keys.ndim == 3 else keys[:m, None]
        v = values[:m] if values.ndim == 3 else values[:m, None]
        x = scale * np.einsum("hd,mhd->hm", q[i], np.broadcast_to(k, (m, H, k.shape[2])))
        top = x.max(axis=1, keepdims=True)
        p = np.exp(x - top)
        l = p.sum(axis=1, keepdims=True)
        L[i] = (top + np.log(l))[:, 0]
        p /= l
        vb = np.broadcast_to(v, (m, H, dv))
        O[i], A[i] = np.einsum("hm,mhd->hd", p, vb), np.einsum("hm,mhd->hd", p, np.abs(vb))
        S[i] = scale * np.einsum("hd,mhd->hm", np.abs(q[i]), np.abs(np.broadcast_to(k, (m, H, k.shape[2])))).max(axis=1)
    return O, L, A, S


def tolerances(O, L, A, S, depth, n_keys, v_top, dtype):
    """What the kernels' arithmetic may be off by.
    Scores: exact products, `depth` additions in fp32, each off by at most 2^-23 of the sum of sizes, then the scaling:
    (depth + 4) 2^-23 S, and 2^-17 for 2^x and subtractions of maxima up to 2^6 (parts joined among them).
    LSE: that, n 2^-24 from the sum, 2^-22 |L|.
    O: a weight is off by delta and by its rounding to the type, half a step (eps / 2), both relative; O is divided by
    the sum of the same rounded weights, so it is a mean with weights off by e = delta + eps / 2 each: at most 2 e / (1 - e)
    of A.  Sums in fp32: n 2^-23 A.  fp16 weights below the normal range are off by 2^-25 against a largest one of at least
    1: n 2^-25 of the largest value.  Then the output's rounding, half a step, or half the type's smallest number."""
    f = torch.finfo(dtype)
    delta = (depth + 4) * 2.0 ** -23 * S + 2.0 ** -17
    lse = delta + n_keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0))
    e = np.minimum(delta + f.eps / 2, 0.5)[..., None]
    o = (2 * e / (1 - e) + n_keys * 2.0 ** -23) * A
    if dtype == torch.float16:
        o = o + n_keys * 2.0 ** -25 * v_top
    return o + (np.abs(O) + o) * f.eps / 2 + f.smallest_normal * f.eps / 2, lse


def check(out, lse, ref, depth, n_keys, v_top, dtype, rows=slice(None)):
    O, L, A, S = (x[rows] for x in ref)
    to, tl = tolerances(O, L, A, S, depth, n_keys, v_top, dtype)
    o, l = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    empty = ~np.isfinite(L)
    assert np.array_equal(l == -math.inf, empty)
    assert np.isfinite(o).all() and (o[empty] == 0).all()
    off = np.abs(l[~empty] - L[~empty])
    assert (off <= tl[~empty]).all(), (off / tl[~empty]).max()
    assert (np.abs(o - O) <= to).all(), (np.abs(o - O) / to).max()
