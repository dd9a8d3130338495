"""Latent attention for torch tensors: keys and values of all heads from one shared latent vector per token.

Argument checks and marshalling over include/fa_latent.h, which defines the operators; the package
re-exports the functions here.

    slots, cu, lens, count, _ = kv_tables_step(new_tokens, lens, block_table, free, count, page_size, T)
    q[..., C:] = latent_cache_append(latent, rope, slots, cache, q_rope, positions, table)   # (or q_out=q[..., C:])
    out, lse = latent_paged_attention_forward(q, cache, block_table, lens, value_dim=C, cu_q=cu, max_q=..., scale=...)

for decoding (the absorbed form: q[..., :C] are queries multiplied by the key projection), and for prompts, with
keys and values projected from the latents,

    out, lse = latent_attention_forward(q, k, k_rope, v, cu_q, cu_k, max_q=..., max_k=...)

What paged.py says of streams, graphs and bad device data holds here too.
"""
from __future__ import annotations

import ctypes
import math

from .paged import _done, _native, _there


class fa_latent_cache(ctypes.Structure):
    """Mirror of `fa_latent_cache` in include/fa_latent.h."""
    _fields_ = [("rows", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("value_dim", ctypes.c_int), ("rope_dim", ctypes.c_int)]


class fa_latent_paged_args(ctypes.Structure):
    """Mirror of `fa_latent_paged_args` in include/fa_latent.h."""
    _fields_ = [("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("cache", fa_latent_cache),
                ("q_stride", ctypes.c_longlong * 2), ("o_stride", ctypes.c_longlong * 2),
                ("T", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


class fa_latent_args(ctypes.Structure):
    """Mirror of `fa_latent_args` in include/fa_latent.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("k_rope", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong * 2), ("k_stride", ctypes.c_longlong * 2), ("v_stride", ctypes.c_longlong * 2),
                ("o_stride", ctypes.c_longlong * 2), ("k_rope_stride", ctypes.c_longlong),
                ("T", ctypes.c_int), ("Tk", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("Dn", ctypes.c_int),
                ("R", ctypes.c_int), ("Dv", ctypes.c_int), ("max_q", ctypes.c_int), ("max_k", ctypes.c_int),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("dtype", ctypes.c_int), ("stream", ctypes.c_void_p)]


def latent_cache_append(latent, rope, slots, cache, q_rope=None, positions=None, table=None, interleaved: bool = False,
                        q_out=None, stream=None, check: bool = False):
    """New tokens' rows (latent, then rope) written into their slots of the cache, in place.

    latent [T, C] and rope [T, R] (None for R = 0) fp16 or bf16, channels contiguous (views of a joint projection are
    fine); slots [T] int32 (kv_tables_step; negative: not stored); cache [num_pages, page_size, C + R] of the same type.
    With positions [T] int32 and table [num_positions, R] (rotary_table) rope is turned first, and q_rope [T, H, R], if given,
    beside it: the result is returned, in q_out (q_rope itself, or a view such as the last R channels of the absorbed
    queries) or a new tensor; None without q_rope.
    """
    if stream is not None:
        with _there(latent, stream):
            return latent_cache_append(latent, rope, slots, cache, q_rope, positions, table, interleaved, q_out, check=check)
    return _done(_native.latent_append(latent, rope, slots, cache, q_rope, positions, table, interleaved, q_out),
                 "fa_latent_cache_append", check, latent)


def latent_paged_attention_forward(q, cache, block_table, lens, value_dim: int, cu_q=None, max_q: int = 1, *, scale: float,
                                   causal: bool = True, out=None, lse=None, workspace=None, stream=None, check: bool = False):
    """O [T, H, value_dim] and LSE [T, H] of absorbed queries q [T, H, C + R] over cached rows: the scores take all channels
    of a row, the values are its first value_dim = C.

    scale has no default: it is the expanded form's, 1/sqrt of the head width there.  cu_q, max_q, lens (the new
    tokens' own included), block_table, causal, given outputs and steps without a query as in paged_attention_forward.
    C <= 512, C + R <= 576, multiples of 8.  A workspace, where one is needed, is allocated unless given.
    """
    if stream is not None:
        with _there(q, stream):
            return latent_paged_attention_forward(q, cache, block_table, lens, value_dim, cu_q, max_q, scale=scale, causal=causal,
                                                  out=out, lse=lse, workspace=workspace, check=check)
    return _done(_native.latent_paged(q, cache, block_table, lens, value_dim, cu_q, max_q, scale, causal, out, lse, workspace),
                 "fa_latent_paged_fwd", check, q)


def latent_attention_forward(q, k, k_rope, v, cu_q, cu_k, max_q: int, max_k: int, scale: float | None = None,
                             causal: bool = True, out=None, lse=None, stream=None, check: bool = False):
    """O [T, H, Dv] and LSE [T, H] of ragged requests: q [T, H, Dn + R] over k [Tk, H, Dn] and k_rope [Tk, R], which all heads
    share, with values v [Tk, H, Dv].

    cu_q, cu_k [B + 1] int32 mark each request's rows of q (at most max_q of them) and of k, k_rope and v (max_k: about the
    most, a hint).  causal: query i of n sees keys j <= i + m - n of its request's m.  Strides are any multiples of 8
    elements, channels contiguous (k and v may be views of one projection).  Dn, Dv <= 128, R <= 64, multiples of 8.
    scale defaults to 1/sqrt(Dn + R).  Rows that are no request's are left as they were.
    """
    if stream is not None:
        with _there(q, stream):
            return latent_attention_forward(q, k, k_rope, v, cu_q, cu_k, max_q, max_k, scale, causal, out, lse, check=check)
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _done(_native.latent_fwd(q, k, k_rope, v, cu_q, cu_k, max_q, max_k, scale, causal, out, lse), "fa_latent_fwd", check, q)
