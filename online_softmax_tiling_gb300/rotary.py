"""Rotary positions for torch tensors: tables, queries and keys turned, and keys turned on their way into
the paged 8-bit cache.

Argument checks and marshalling over include/fa_rotary.h, which defines the operators; the package
re-exports the functions here.

    table = rotary_table(max_positions, *rotary_frequencies(128))
    q, k = rotary_embed(q, k, positions, table)
    q = kv_cache_append_rotary(q, k, v, positions, table, slots, k_cache, v_cache, k_scale, v_scale)

The second call turns and returns, the third replaces it and kv_cache_append (by one launch for a decode step, by two
where there are many queries).  What
paged.py says of streams, graphs and bad device data holds here too.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .paged import _done, _native, _there


class fa_rotary(ctypes.Structure):
    """Mirror of `fa_rotary` in include/fa_rotary.h."""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("num_positions", ctypes.c_int),
                ("dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int)]


class fa_rotary_part(ctypes.Structure):
    """Mirror of `fa_rotary_part` in include/fa_rotary.h."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("x_stride", ctypes.c_longlong * 2),
                ("y_stride", ctypes.c_longlong * 2), ("heads", ctypes.c_int)]


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """(w, factor): the angles per position w_i = base^(-2 i / dim) of the dim / 2 pairs (float64, on the CPU), and
    what cosines and sines are multiplied by.

    scaling, for contexts `factor` times longer than `original_length`:
      None        none
      "linear"    every w_i divided by factor
      "base"      base raised to base * factor^(dim / (dim - 2)): the slowest pair is divided by factor, the fastest stays
      "bands"     pairs of fewer than slow_turns turns within original_length divided by factor, those of more than
                  fast_turns left, between them a ramp over the pair's index (the two limits rounded outwards to whole
                  pairs); comes with the factor 0.1 ln(factor) + 1
    """
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and positive")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("base must be positive, factor at least 1")
    i = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == "base":
        if dim < 4:
            raise ValueError('scaling "base" needs at least two pairs')
        base = base * factor ** (dim / (dim - 2))
    w = base ** (-2.0 * i / dim)
    if scaling in (None, "base"):
        return w, 1.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling != "bands":
        raise ValueError(f"unknown scaling {scaling!r}")
    if original_length is None or original_length < 1 or not fast_turns > slow_turns > 0 or base <= 1:
        raise ValueError('scaling "bands" needs original_length, fast_turns > slow_turns > 0 and base > 1')
    at = [dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (fast_turns, slow_turns)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
    keep = 1.0 - ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return w / factor * (1.0 - keep) + w * keep, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def rotary_table(num_positions: int, frequencies, factor: float = 1.0, device="cuda"):
    """[num_positions, dim] float32: the cosines of position * w_i, then the sines, times factor; angles and functions
    in 64 bits (a far position's angle keeps its fraction of a turn)."""
    if num_positions < 1:
        raise ValueError("num_positions must be at least 1")
    w = frequencies.to(device=device, dtype=torch.float64)
    if w.dim() != 1:
        raise ValueError("frequencies must be [dim / 2]")
    out = torch.empty((num_positions, 2 * w.numel()), dtype=torch.float32, device=device)
    step = max(1, (1 << 24) // max(1, w.numel()))  # (the angles in 64 bits take no more than a few hundred MB)
    for p in range(0, num_positions, step):
        n = min(step, num_positions - p)
        a = torch.arange(p, p + n, dtype=torch.float64, device=device)[:, None] * w
        out[p:p + n, :w.numel()] = torch.cos(a) * factor
        out[p:p + n, w.numel():] = torch.sin(a) * factor
    return out


def rotary_embed(q, k, positions, table, interleaved: bool = False, inverse: bool = False, q_out=None, k_out=None,
                 stream=None, check: bool = False):
    """(q, k) with the first table.shape[1] channels of every head turned by the tokens' positions.

    q [T, Hq, d] and k [T, Hk, d] (or None) fp16 or bf16, any token and head strides that are multiples of 8 elements,
    d contiguous and a multiple of 8 (views of a joint projection are fine); positions [T] int32, rows of table
    [num_positions, dim] float32 (rotary_table); dim a multiple of 16.  interleaved: pairs (2 i, 2 i + 1) instead of (i, i + dim / 2).  A
    negative position leaves its token as it is; so does one beyond the table, which fa_check_device_status
    reports.  inverse turns back: the gradient with respect to q and k, given that of the outputs (as everywhere in this
    package nothing is recorded for autograd, whatever q and k require: a backward pass makes that call itself).  q_out, k_out: q and k
    themselves (in place), or tensors that do not overlap them; new ones unless given.
    """
    if stream is not None:
        with _there(q, stream):
            return rotary_embed(q, k, positions, table, interleaved, inverse, q_out, k_out, check=check)
    return _done(_native.rotary_embed(q, k, positions, table, interleaved, inverse, q_out, k_out), "fa_rotary_embed", check, q)


def kv_cache_append_rotary(q, k, v, positions, table, slots, k_cache, v_cache, k_scale, v_scale, k_bounds=None,
                           interleaved: bool = False, q_out=None, stream=None, check: bool = False):
    """kv_cache_append of keys turned on their way (a key is rounded once, to the cache's 8 bits), and the
    queries [T, Hq, d] turned as rotary_embed does, in the same launch or, where there are many, in one of their own behind
    it.  Returns the turned queries (q_out if given, which may be q; None for q None)."""
    if stream is not None:
        with _there(k, stream):
            return kv_cache_append_rotary(q, k, v, positions, table, slots, k_cache, v_cache, k_scale, v_scale, k_bounds,
                                          interleaved, q_out, check=check)
    return _done(_native.append_rotary(q, k, v, positions, table, slots, k_cache, v_cache, k_scale, v_scale, k_bounds,
                                       interleaved, q_out), "fa_kv_cache_append_rotary", check, k)
