"""Paged attention of no queries through the C ABI, on the host: what empty tensors have for addresses (NULL)
is taken, what else is wrong with the call is still refused.  Fake addresses, as in test_paged_abi.py, so
only in a process that sees no GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

import online_softmax_tiling_gb300 as fa
from tests.test_abi import GPU_VISIBLE, ROOT
from tests.test_paged_abi import A, BAD, MISAL, _args, _cache, lib  # noqa: F401 (lib: the fixture)

NONE = dict(T=0, q=None, o=None, lse=None)


def test_runs_where_no_gpu_is_visible():
    if not GPU_VISIBLE:
        pytest.skip("no GPU visible: the tests below run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", __file__],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.mark.parametrize("kw,want", [
    (dict(cu_q=A), 0), (dict(cu_q=A, max_q=0), 0), (dict(cu_q=A, max_q=90, num_splits=5), 0),
    (dict(cu_q=A, Hq=64, num_splits=0), 0),
    (dict(B=0), 0), (dict(B=0, max_q=0, block_table=None, lens=None), 0), (dict(B=0, cu_q=A), 0),
    (dict(B=0, num_splits=0), 0), (dict(B=0, selected_count=A, num_selected=2), 0),
    (dict(), BAD), (dict(B=-1, cu_q=A), BAD), (dict(cu_q=A, lens=None), BAD), (dict(cu_q=A, block_table=None), BAD),
    (dict(cu_q=A, max_q=-1), BAD), (dict(cu_q=A, scale=0.0), BAD), (dict(cu_q=A, Hq=3), BAD), (dict(cu_q=A, dtype=7), BAD),
    (dict(cu_q=A, max_pages=0), BAD), (dict(cu_q=A, cache=_cache(k=None)), BAD), (dict(cu_q=A, q=A + 8), MISAL)])
def test_calls_without_a_query(lib, kw, want):  # noqa: F811
    a = _args(**{**NONE, **kw})
    assert lib.fa_paged_fwd(ctypes.addressof(a)) == want
    assert lib.fa_paged_num_splits(ctypes.addressof(a)) == 1
    assert lib.fa_paged_workspace_size(ctypes.addressof(a)) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(o=None), dict(lse=None), dict(B=0), dict(cu_q=A, max_q=0),
                                dict(selected_count=A, num_selected=2)])
def test_calls_with_queries_are_refused_as_before(lib, kw):  # noqa: F811
    assert lib.fa_paged_fwd(ctypes.addressof(_args(**kw))) == BAD
