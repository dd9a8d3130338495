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
captured in a CUDA graph (after one call outside of a capture).  Bad device
data (a page or slot outside of the cache, lengths beyond the table) is
skipped by the kernels and reported by fa_check_device_status, which
check=True calls here.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import (FA_BF16, FA_FP16, FA_OK, FaError, _checked, library)

FA_ERR_NO_PAGES = 6
FA_PAGED_MAX_SPLITS = 64
_E4M3, _F32, _I32, _I8 = torch.float8_e4m3fn, torch.float32, torch.int32, torch.int8
_CODES = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


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


# The same structures packed in one step (a Structure filled field by field
# costs several times as much on the host).
_PACK_CACHE = struct.Struct("@5P4i")
_PACK_ARGS = struct.Struct("@8P5P4i4q6if3iPNP")
_PACK_STRIDE = struct.Struct("@2q")


def _fail(name, t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    raise ValueError(f"{name} must be {what}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _need(name, t, dtype, shape, dev):
    """Address of t: contiguous, of this type and shape, on CUDA device number `dev`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _fail(name, t, f"a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _rows16(name, t, dev, dtype):
    """Strides of t: [rows, heads, d] of a 16-bit type with contiguous d."""
    if t.dim() != 3 or t.get_device() != dev or t.dtype is not dtype:
        _fail(name, t, f"a {dtype} tensor [tokens, heads, d] on cuda:{dev}")
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.shape[2] > 1:
        _fail(name, t, "a tensor with a contiguous last dimension")
    if s0 < 8 or s1 < 8:
        # the stride of a dimension of at most one element is never used: any valid one will do
        n, h, _ = t.shape
        return (s0 if n > 1 else 8), (s1 if h > 1 else 8)
    return s0, s1


def _dtype_of(t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float16 or bfloat16)")
    return code


def _device_of(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    return dev


class _there:
    """Makes CUDA device `dev` and `stream` (a torch stream, a handle or None) the current ones."""

    def __init__(self, dev, stream):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
        self.contexts = [torch.cuda.device(dev)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *a):
        for c in reversed(self.contexts):
            c.__exit__(*a)


def _cache_sizes(k_cache):
    if k_cache.dim() != 4:
        _fail("k_cache", k_cache, "[num_pages, Hk, page_size, d]")
    return k_cache.shape


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
    nothing and its slots are all -1.  check=True waits for it and raises.
    """
    device = _device_of(new_tokens)
    if stream is not None or device != _current_device():
        with _there(device, stream):
            return kv_tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size,
                                  max_tokens, check=check)
    if block_table.dim() != 2 or new_tokens.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("new_tokens [B], block_table [B, max_pages], free_pages [capacity]")
    B, M = block_table.shape
    handle = _raw_stream(device)
    max_tokens = int(max_tokens)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    out = new_tokens.new_empty(max_tokens + 2 * B + 3, dtype=_I32)
    at = out.data_ptr()
    at_cu = at + 4 * max_tokens
    at_lens = at_cu + 4 * (B + 1)
    st = library().fa_kv_tables_step(
        _need("new_tokens", new_tokens, _I32, (B,), device), _need("lens", lens, _I32, (B,), device),
        _need("block_table", block_table, _I32, (B, M), device),
        _need("free_pages", free_pages, _I32, free_pages.shape, device),
        _need("free_count", free_count, _I32, (1,), device), B, M, free_pages.shape[0], page_size,
        max_tokens, at, at_cu, at_lens, at_lens + 4 * B, at_lens + 4 * B + 4, handle)
    if st != FA_OK:
        raise FaError(st, "fa_kv_tables_step")
    parts = out.split_with_sizes((max_tokens, B + 1, B, 1, 1))
    if check:
        _checked(handle, "fa_kv_tables_step")
        code = int(parts[4].item())
        if code != FA_OK:
            raise FaError(code, "fa_kv_tables_step")
    return parts


def kv_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds=None, stream=None,
                    check: bool = False):
    """Quantise new keys and values into their slots of the cache, in place.

    k, v [T, Hk, d] fp16 or bf16 (any token and head strides that are multiples
    of 8 elements, d contiguous); slots [T] int32 (kv_tables_step; negative
    rows are not stored); k_cache, v_cache [num_pages, Hk, page_size, d]
    float8_e4m3fn; k_scale, v_scale [num_pages, Hk] float32; k_bounds
    [num_pages, Hk, 2, d] int8 for kv_page_select.  The tokens of one page must
    be consecutive rows with ascending slots.
    """
    device = _device_of(k)
    if stream is not None or device != _current_device():
        with _there(device, stream):
            return kv_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds,
                                   check=check)
    shape = _cache_sizes(k_cache)
    N, Hk, P, d = shape
    dtype = _dtype_of(k)
    ks, vs = _rows16("k", k, device, k.dtype), _rows16("v", v, device, k.dtype)
    T = k.shape[0]
    if k.shape != (T, Hk, d) or v.shape != (T, Hk, d):
        raise ValueError(f"k and v must be [T, {Hk}, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    cache = _PACK_CACHE.pack(
        _need("k_cache", k_cache, _E4M3, shape, device), _need("v_cache", v_cache, _E4M3, shape, device),
        _need("k_scale", k_scale, _F32, (N, Hk), device), _need("v_scale", v_scale, _F32, (N, Hk), device),
        0 if k_bounds is None else _need("k_bounds", k_bounds, _I8, (N, Hk, 2, d), device), N, P, Hk, d)
    at = _need("slots", slots, _I32, (T,), device)
    if T == 0:
        return
    handle = _raw_stream(device)
    st = library().fa_kv_cache_append(cache, k.data_ptr(), v.data_ptr(), at, T, _PACK_STRIDE.pack(*ks),
                                      _PACK_STRIDE.pack(*vs), dtype, handle)
    if st != FA_OK:
        raise FaError(st, "fa_kv_cache_append")
    if check:
        _checked(handle, "fa_kv_cache_append")


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
    (0: chosen by the library); a workspace, where the count needs one, is
    allocated unless given.  Rows of given outputs behind the last query are
    left as they were.  A kernel whose waits run out (2 s) leaves outputs
    unwritten and reports it through fa_check_device_status, as in
    attention_forward.
    """
    device = _device_of(q)
    if stream is not None or device != _current_device():
        with _there(device, stream):
            return paged_attention_forward(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_q,
                                           max_q, scale, causal, selected, selected_count, out, lse,
                                           num_splits, workspace, check=check)
    shape = _cache_sizes(k_cache)
    N, Hk, P, d = shape
    dtype = _dtype_of(q)
    qs = _rows16("q", q, device, q.dtype)
    T, Hq, dq = q.shape
    if dq != d or block_table.dim() != 2:
        raise ValueError("q must be [T, Hq, d] with the cache's d, block_table [B, max_pages]")
    B, M = block_table.shape
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        os = (Hq * d, d)
    else:
        os = _rows16("out", out, device, q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    if lse is None:
        lse = q.new_empty((T, Hq), dtype=_F32)
        at_lse = lse.data_ptr()
    else:
        at_lse = _need("lse", lse, _F32, (T, Hq), device)
    keep = at_sel = at_count = 0
    if selected is not None:
        if selected_count is None or selected.dim() != 3:
            raise ValueError("selected [B, Hk, keep] comes with selected_count [B, Hk]")
        keep = selected.shape[2]
        at_sel = _need("selected", selected, _I32, (B, Hk, keep), device)
        at_count = _need("selected_count", selected_count, _I32, (B, Hk), device)
    elif selected_count is not None:
        raise ValueError("selected_count comes with selected")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    handle = _raw_stream(device)
    fields = (q.data_ptr(), out.data_ptr(), at_lse,
              0 if cu_q is None else _need("cu_q", cu_q, _I32, (B + 1,), device),
              _need("block_table", block_table, _I32, (B, M), device), _need("lens", lens, _I32, (B,), device),
              at_sel, at_count,
              _need("k_cache", k_cache, _E4M3, shape, device), _need("v_cache", v_cache, _E4M3, shape, device),
              _need("k_scale", k_scale, _F32, (N, Hk), device), _need("v_scale", v_scale, _F32, (N, Hk), device),
              0, N, P, Hk, d, *qs, *os, T, B, Hq, max_q, M, keep, scale, causal, dtype, num_splits)
    lib = library()
    args = _PACK_ARGS.pack(*fields, 0, 0, handle)
    nbytes = lib.fa_paged_workspace_size(args)
    if nbytes:
        if workspace is None:
            workspace = q.new_empty(nbytes, dtype=torch.uint8)
        elif workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
        args = _PACK_ARGS.pack(*fields, workspace.data_ptr(), workspace.nbytes, handle)
    st = lib.fa_paged_fwd(args)
    if st != FA_OK:
        raise FaError(st, "fa_paged_fwd")
    if check:
        _checked(handle, "fa_paged_fwd")
    return out, lse


def kv_page_select(q, k_bounds, k_scale, block_table, lens, page_size: int, num_selected: int,
                   stream=None, check: bool = False):
    """(selected [B, Hk, num_selected], selected_count [B, Hk]) int32: the pages
    of each key head that one query per request q [B, Hq, d] should read, by the
    exact whole-number score of include/fa_paged.h over k_bounds
    [num_pages, Hk, 2, d]; ascending, -1 behind the last, the last token's page
    always among them."""
    device = _device_of(q)
    if stream is not None or device != _current_device():
        with _there(device, stream):
            return kv_page_select(q, k_bounds, k_scale, block_table, lens, page_size, num_selected,
                                  check=check)
    dtype = _dtype_of(q)
    qs = _rows16("q", q, device, q.dtype)
    if k_bounds.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_bounds [num_pages, Hk, 2, d], block_table [B, max_pages]")
    N, Hk, _, d = k_bounds.shape
    B, M = block_table.shape
    Hq = q.shape[1]
    num_selected = int(num_selected)
    if q.shape != (B, Hq, d) or num_selected < 1:
        raise ValueError("q must be [B, Hq, d], num_selected at least 1")
    cache = _PACK_CACHE.pack(0, 0, _need("k_scale", k_scale, _F32, (N, Hk), device), 0,
                             _need("k_bounds", k_bounds, _I8, (N, Hk, 2, d), device), N, page_size, Hk, d)
    selected, count = lens.new_empty((B, Hk, num_selected), dtype=_I32), lens.new_empty((B, Hk), dtype=_I32)
    handle = _raw_stream(device)
    st = library().fa_kv_page_select(
        cache, q.data_ptr(), _PACK_STRIDE.pack(*qs), _need("block_table", block_table, _I32, (B, M), device),
        _need("lens", lens, _I32, (B,), device), B, Hq, M, num_selected, dtype, selected.data_ptr(),
        count.data_ptr(), handle)
    if st != FA_OK:
        raise FaError(st, "fa_kv_page_select")
    if check:
        _checked(handle, "fa_kv_page_select")
    return selected, count
