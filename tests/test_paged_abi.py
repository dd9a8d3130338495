"""The refusals of include/fa_paged.h's entry points and of their Python wrappers, on the host.

As in test_abi.py the C calls pass fake addresses that are never dereferenced, so they run only
in a process that sees no GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

import online_softmax_tiling_gb300 as fa
from tests.test_abi import GPU_VISIBLE, ROOT

A = 0x10000
BAD, UNSUP, MISAL, CUDA = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED, fa.FA_ERR_CUDA


def test_runs_where_no_gpu_is_visible():
    if not GPU_VISIBLE:
        pytest.skip("no GPU visible: the tests below run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", __file__],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.fixture()
def lib():
    if GPU_VISIBLE:
        pytest.skip("run in a child process that sees no GPU")
    if not os.path.exists(fa.LIBRARY):
        from online_softmax_tiling_gb300 import build
        build.build()
    return fa.library()


def _cache(**kw):
    c = fa.fa_kv_cache(A, A + 0x1000, A + 0x2000, A + 0x3000, A + 0x4000, 10, 16, 2, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_REFUSALS = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD),
    (dict(num_pages=0), BAD), (dict(page_size=8), BAD), (dict(page_size=48), BAD), (dict(page_size=256), BAD),
    (dict(Hk=0), BAD), (dict(d=0), UNSUP), (dict(d=24), UNSUP), (dict(d=272), UNSUP),
    (dict(num_pages=1 << 30), BAD), (dict(k=A + 8), MISAL), (dict(v=A + 1), MISAL), (dict(k_scale=A + 2), MISAL),
    (dict(k_bounds=A + 4), MISAL)]


def _args(cache=None, **kw):
    a = fa.fa_paged_args()
    a.q, a.o, a.lse, a.block_table, a.lens = A, A + 0x100, A + 0x200, A + 0x300, A + 0x400
    a.cache = cache or _cache()
    a.q_stride[:] = a.o_stride[:] = [256, 64]
    a.T = a.B = 3
    a.Hq, a.max_q, a.max_pages, a.scale, a.causal, a.dtype, a.num_splits = 4, 1, 20, 0.125, 1, fa.FA_BF16, 1
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def _fwd(lib, a):
    return lib.fa_paged_fwd(ctypes.addressof(a))


@pytest.mark.parametrize("kw,want", CACHE_REFUSALS)
def test_cache_refusals(lib, kw, want):
    c = _cache(**kw)
    assert _fwd(lib, _args(c)) == want
    st = (ctypes.c_longlong * 2)(128, 64)
    p = ctypes.addressof
    assert lib.fa_kv_cache_append(p(c), A, A, A, 5, p(st), p(st), fa.FA_FP16, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(block_table=None), BAD),
    (dict(lens=None), BAD), (dict(B=0), BAD), (dict(T=-1), BAD), (dict(T=4), BAD), (dict(max_q=2), BAD),
    (dict(cu_q=A, max_q=0), BAD), (dict(Hq=3), BAD), (dict(Hq=0), BAD), (dict(max_pages=0), BAD),
    (dict(max_pages=(1 << 26) + 1), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(dtype=2), BAD),
    (dict(num_splits=-1), BAD), (dict(num_splits=65), BAD), (dict(num_splits=3), BAD), (dict(num_splits=16), CUDA),
    (dict(selected=A), BAD), (dict(selected_count=A), BAD), (dict(selected=A, selected_count=A), BAD),
    (dict(selected=A, selected_count=A, num_selected=2, cu_q=A, max_q=2), BAD),
    (dict(q=A + 8), MISAL), (dict(o=A + 8), MISAL), (dict(lse=A + 2), MISAL), (dict(cu_q=A + 1, max_q=1), MISAL),
    (dict(q_stride=[0, 64]), MISAL), (dict(q_stride=[256, 60]), MISAL), (dict(o_stride=[-256, 64]), MISAL),
    (dict(), CUDA), (dict(T=0, cu_q=A), 0), (dict(num_splits=5, workspace=A + 16, workspace_bytes=1 << 30), MISAL),
    (dict(num_splits=5, workspace=A, workspace_bytes=3 * 4 * 5 * 65 * 4 - 1), BAD),
    (dict(num_splits=5, workspace=A, workspace_bytes=3 * 4 * 5 * 65 * 4), CUDA)])
def test_attention_refusals(lib, kw, want):
    assert _fwd(lib, _args(**kw)) == want


def test_null_structures(lib):
    assert lib.fa_paged_fwd(None) == BAD
    assert lib.fa_kv_cache_append(None, A, A, A, 1, A, A, 0, None) == BAD
    assert lib.fa_paged_num_splits(None) == 1
    assert lib.fa_kv_page_select(None, A, A, A, A, 1, 1, 1, 1, 0, A, A, None) == BAD


def test_splits_and_workspace(lib):
    """With GB300's 152 SMs (counted where no device answers)."""
    def n(**kw):
        a = _args(**kw)  # (held until the call is over)
        return lib.fa_paged_num_splits(ctypes.addressof(a))

    def ws(**kw):
        a = _args(**kw)
        return lib.fa_paged_workspace_size(ctypes.addressof(a))

    assert n(max_pages=16) == 1                                   # 256 keys: one range
    assert 1 < n(max_pages=1000) <= fa.FA_PAGED_MAX_SPLITS        # 6 units, many keys
    assert n(T=4000, B=4000, max_pages=1000) == 1                 # units enough
    assert n(scale=-1.0) == 1
    for s in (1, 2, 4, 8, 16):                                    # joined on chip
        assert ws(num_splits=s) == 0
    assert ws(num_splits=3) == 3 * 4 * 3 * 64 * 4 + 3 * 4 * 3 * 4
    assert ws(num_splits=3, scale=-1.0) == 0 and lib.fa_paged_workspace_size(None) == 0
    rows = dict(cu_q=A, T=100, max_q=90, num_splits=4)            # prompt rows: through a workspace
    assert ws(**rows) == 100 * 4 * 4 * 64 * 4 + 100 * 4 * 4 * 4


@pytest.mark.parametrize("requests,want", [(1, 8), (7, 8), (8, 4), (18, 4), (19, 2), (38, 2), (76, 1), (200, 2), (2000, 1)])
def test_ranges_fill_one_wave_of_clusters(lib, requests, want):
    """Two heads and 2048 keys: as many key ranges as leave every cluster a place on the 152 SMs."""
    a = _args(T=requests, B=requests, max_pages=128)
    assert lib.fa_paged_num_splits(ctypes.addressof(a)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), BAD), (dict(slots=None), BAD), (dict(T=-1), BAD), (dict(dtype=5), BAD), (dict(k=A + 8), MISAL),
    (dict(ks=(128, 60)), MISAL), (dict(vs=(0, 64)), MISAL), (dict(slots=A + 1), MISAL), (dict(T=0), 0), (dict(T=(1 << 30) + 1), BAD), (dict(), CUDA)])
def test_append_refusals(lib, kw, want):
    a = dict(k=A, v=A, slots=A, T=5, ks=(128, 64), vs=(128, 64), dtype=fa.FA_BF16)
    a.update(kw)
    c, ks, vs = _cache(), (ctypes.c_longlong * 2)(*a["ks"]), (ctypes.c_longlong * 2)(*a["vs"])
    assert lib.fa_kv_cache_append(ctypes.addressof(c), a["k"], a["v"], a["slots"], a["T"], ctypes.addressof(ks),
                                  ctypes.addressof(vs), a["dtype"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(new=None), BAD), (dict(B=0), BAD), (dict(B=16385), UNSUP), (dict(M=0), BAD), (dict(F=0), BAD),
    (dict(P=20), BAD), (dict(T=-1), BAD), (dict(slots=None), BAD), (dict(lens_out=A + 4), BAD),
    (dict(count_out=A + 16), BAD), (dict(M=1 << 28), BAD), (dict(table=A + 2), MISAL), (dict(), CUDA)])
def test_tables_refusals(lib, kw, want):
    a = dict(new=A, lens=A + 4, table=A + 8, free=A + 12, count=A + 16, B=4, M=5, F=6, P=16, T=7, slots=A + 20,
             cu=A + 24, lens_out=A + 28, count_out=A + 32, status=A + 36)
    a.update(kw)
    assert lib.fa_kv_tables_step(a["new"], a["lens"], a["table"], a["free"], a["count"], a["B"], a["M"], a["F"], a["P"],
                                 a["T"], a["slots"], a["cu"], a["lens_out"], a["count_out"], a["status"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(B=0), BAD), (dict(Hq=3), BAD), (dict(M=0), BAD), (dict(M=32769), UNSUP),
    (dict(keep=0), BAD), (dict(dtype=3), BAD), (dict(q=A + 8), MISAL), (dict(sel=A + 1), MISAL),
    (dict(cache=dict(k_bounds=None)), BAD), (dict(cache=dict(k_scale=None)), BAD), (dict(cache=dict(d=20)), UNSUP),
    (dict(Hq=2 * 1000, cache=dict(d=256)), UNSUP), (dict(cache=dict(k=None, v=None, v_scale=None)), CUDA), (dict(), CUDA)])
def test_select_refusals(lib, kw, want):
    a = dict(q=A, B=2, Hq=4, M=10, keep=3, dtype=fa.FA_FP16, sel=A, count=A, cache={})
    a.update(kw)
    c, st = _cache(**a["cache"]), (ctypes.c_longlong * 2)(512, 64)
    assert lib.fa_kv_page_select(ctypes.addressof(c), a["q"], ctypes.addressof(st), A, A, a["B"], a["Hq"], a["M"],
                                 a["keep"], a["dtype"], a["sel"], a["count"], None) == want


def test_wrappers_refuse_tensors_on_the_cpu():
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, b = torch.ones((3, 2)), torch.zeros((3, 2, 2, 64), dtype=torch.int8)
    q = torch.zeros((4, 2, 64), dtype=torch.float16)
    table = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: fa.kv_tables_step(i, i, table, i, i[:1], 16, 8),
                 lambda: fa.kv_cache_append(q, q, i, c, c, s, s),
                 lambda: fa.paged_attention_forward(q, c, c, s, s, table, i),
                 lambda: fa.kv_page_select(q, b, s, table, i, 16, 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fa.kv_tables_step(None, i, table, i, i[:1], 16, 8)
