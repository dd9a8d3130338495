"""Serving operators around a paged key/value cache held in 8 bits, for torch tensors.

Argument checks and marshalling over include/fa_paged.h, which defines every
operator, format and status; the package re-exports the functions here.

    slots, cu, lens, count, status = kv_tables_step(new_tokens, lens, table, free, count, ...)
    kv_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    out, lse = paged_attention_forward(q, k_cache, v_cache, k_scale, v_scale, table, lens,
                                       cu_q=cu, max_q=...)

and, for one query per request over the best pages of a long context,

    selected, count = kv_page_select(q, k_bounds, k_scale, table, lens, page_size, keep)
    out, lse = paged_attention_forward(..., selected=selected, selected_count=count)

All work is enqueued on `stream` (default: torch's current stream of the
tensors' device); outputs and workspaces that are not given are allocated on
that stream.  Nothing is allocated inside the library, so every call can be
captured in a CUDA graph (after one call of the same sizes outside of a capture).  Bad device
data (a page or slot outside of the cache, lengths beyond the table) is
skipped by the kernels and reported by fa_check_device_status, which
check=True calls here.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import sysconfig

import torch

from . import FA_OK, FaError, _checked, library

FA_ERR_NO_PAGES = 6
FA_PAGED_MAX_SPLITS = 64


class fa_kv_cache(ctypes.Structure):
    """Mirror of `fa_kv_cache` in include/fa_paged.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_bounds", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int)]


class fa_paged_args(ctypes.Structure):
    """Mirror of `fa_paged_args` in include/fa_paged.h."""
    _fields_ = [("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("cu_q", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("selected", ctypes.c_void_p), ("selected_count", ctypes.c_void_p),
                ("cache", fa_kv_cache),
                ("q_stride", ctypes.c_longlong * 2), ("o_stride", ctypes.c_longlong * 2),
                ("T", ctypes.c_int), ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("num_selected", ctypes.c_int),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
                ("num_splits", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


def _load():
    """The compiled binding (csrc/torch_binding.cpp) beside the library it calls."""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.path.join(here, "_paged_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    library()  # (raises, saying how to build, if that is missing)
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m online_softmax_tiling_gb300.build`")
    spec = importlib.util.spec_from_file_location("online_softmax_tiling_gb300._paged_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_native = _load()


class _there:
    """Makes the device of `t` and `stream` (a torch stream or a handle) the current ones."""

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=t.device)
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        self.contexts = (torch.cuda.device(t.device), torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *a):
        for c in reversed(self.contexts):
            c.__exit__(*a)


def _done(result, what, check, t):
    """The outputs of a call, or its error; check=True also waits for the kernels' status."""
    if type(result) is int:
        raise FaError(result, what)
    if check:
        with torch.cuda.device(t.device):
            _checked(torch.cuda.current_stream().cuda_stream, what)
    return result


def kv_tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size: int,
                   max_tokens: int, stream=None, check: bool = False):
    """One step's bookkeeping of B requests: (slots, cu_new, lens_out, free_count_out, status).

    new_tokens [B] int32: tokens to add to each request (negative: it ends and
    its pages are released); lens [B] int32: tokens held; block_table
    [B, max_pages] int32 and free_pages [capacity] int32 are updated in place;
    free_count [1] int32.  slots [max_tokens], cu_new [B + 1], lens_out [B],
    free_count_out [1] and status [1] are new int32 tensors: the next step
    takes lens_out and free_count_out.  status is FA_OK, FA_ERR_NO_PAGES or
    FA_ERR_INVALID_ARG on the device; unless it is FA_OK the step changed
    nothing and its slots are all -1.  A page number that cannot be gives its
    tokens slot -1 and is reported by fa_check_device_status.  check=True waits
    for both and raises.
    """
    if stream is not None:
        with _there(new_tokens, stream):
            return kv_tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size,
                                  max_tokens, check=check)
    out = _done(_native.tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size, max_tokens),
                "fa_kv_tables_step", check, new_tokens)
    if check and out[4].item() != FA_OK:
        raise FaError(out[4].item(), "fa_kv_tables_step")
    return out


def kv_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds=None, stream=None,
                    check: bool = False):
    """Quantise new keys and values into their slots of the cache, in place.

    k, v [T, Hk, d] fp16 or bf16 (any token and head strides that are multiples
    of 8 elements, d contiguous); slots [T] int32 (kv_tables_step; negative
    rows are not stored); k_cache, v_cache [num_pages, Hk, page_size, d]
    float8_e4m3fn; k_scale, v_scale [num_pages, Hk] float32; k_bounds
    [num_pages, Hk, 2, d] int8 for kv_page_select.  The tokens of one page must
    follow one another with slots ascending by one; rows that are not stored may
    stand between them, fewer than 128 in a row.  Any other order within a page is
    reported by fa_check_device_status and not stored.
    """
    if stream is not None:
        with _there(k, stream):
            return kv_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds, check=check)
    _done(_native.append(k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds), "fa_kv_cache_append", check, k)


def paged_attention_forward(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_q=None,
                            max_q: int = 1, scale: float | None = None, causal: bool = True,
                            selected=None, selected_count=None, out=None, lse=None,
                            num_splits: int = 0, workspace=None, stream=None, check: bool = False):
    """O [T, Hq, d] and LSE [T, Hq] of new queries q [T, Hq, d] over cached keys.

    cu_q [B + 1] int32 marks each request's rows of q (at most max_q of them);
    without it there is one query per request.  lens [B] int32 counts each
    request's keys, the new tokens' included; block_table [B, max_pages] int32.
    causal: query i of n sees keys j <= i + len - n.  selected [B, Hk, keep]
    with selected_count [B, Hk] (kv_page_select) restricts every key head to
    those pages.  scale defaults to 1/sqrt(d).  num_splits: key ranges per row
    (0: chosen by the library from the table's width); a workspace, where the count needs one, is
    allocated unless given.  Rows of given outputs before the first query and
    behind the last are left as they were.  A step without a query (T = 0, any
    number of requests) returns empty outputs.  A kernel whose waits run out (2 s) leaves outputs
    undefined and reports it through fa_check_device_status, as in
    attention_forward.
    """
    if stream is not None:
        with _there(q, stream):
            return paged_attention_forward(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_q,
                                           max_q, scale, causal, selected, selected_count, out, lse,
                                           num_splits, workspace, check=check)
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _done(_native.attend(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_q, max_q, scale, causal,
                                selected, selected_count, out, lse, num_splits, workspace),
                 "fa_paged_fwd", check, q)


def kv_page_select(q, k_bounds, k_scale, block_table, lens, page_size: int, num_selected: int,
                   stream=None, check: bool = False):
    """(selected [B, Hk, num_selected], selected_count [B, Hk]) int32: the pages
    of each key head that one query per request q [B, Hq, d] should read, by the
    exact whole-number score of include/fa_paged.h over k_bounds
    [num_pages, Hk, 2, d]; ascending, -1 behind the last, the last token's page
    always among them.  Empty for B = 0."""
    if stream is not None:
        with _there(q, stream):
            return kv_page_select(q, k_bounds, k_scale, block_table, lens, page_size, num_selected, check=check)
    return _done(_native.page_select(q, k_bounds, k_scale, block_table, lens, page_size, num_selected),
                 "fa_kv_page_select", check, q)
