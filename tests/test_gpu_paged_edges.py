"""The paged-cache operators (include/fa_paged.h) on the GPU at the edges of what their documentation
allows: steps without a query, marks that begin behind row 0, page numbers that cannot be, slots left
out, pending statuses."""
import math

import numpy as np
import pytest

from tests import paged_ref as ref
from tests import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from online_softmax_tiling_gb300 import build
    build.build()
    yield


_torch, _fa, _i32, _ok = base._torch, base._fa, base._i32, base._ok


# ------------------------------------------------- marks behind row 0
@pytest.mark.parametrize("Hk,G,d,news", [(2, 4, 128, [3, 2, 1]), (2, 4, 64, [200, 70, 1]), (1, 4, 256, [90, 40, 2])])
@pytest.mark.parametrize("splits", [1, 2, 3, 5])
def test_rows_before_the_first_query_are_left(Hk, G, d, news, splits):
    """The later requests of a batch alone (a view of its marks): rows of the earlier one stay as they were."""
    torch, fa = _torch(), _fa()
    case = base._attend_case([n + 300 for n in news], news, Hk, G, 16, d, "bf16", 211 + d)
    cache, table, lens, cu, q = case
    g, marks = cache.cuda(), _i32(cu)
    out = torch.full_like(q, 7.0, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    fa.paged_attention_forward(q.cuda(), *g[:4], _i32(table)[1:], _i32(lens)[1:], cu_q=marks[1:], max_q=max(news),
                               out=out, lse=lse, num_splits=splits)
    _ok()
    n = news[0]
    assert (out[:n] == 7).all() and (lse[:n] == 7).all()
    base._check_attend(case, out, lse, rows=slice(n, None))


# ------------------------------------------------- steps without a query
@pytest.mark.parametrize("d", [64, 256])
def test_attention_of_no_queries(d):
    """A step that brings no query: empty outputs, given ones left alone, nothing launched."""
    torch, fa = _torch(), _fa()
    cache, table, lens, cu, q = base._attend_case([40, 90], [1, 1], 2, 2, 16, d, "bf16", 201)
    g, dev = cache.cuda(), (_i32(table), _i32(lens))
    none = q[:0].cuda()
    for max_q in (0, 1, 100):
        out, lse = fa.paged_attention_forward(none, *g[:4], *dev, cu_q=_i32([0, 0, 0]), max_q=max_q, check=True)
        assert out.shape == (0, 4, d) and lse.shape == (0, 4) and out.dtype == q.dtype
    o, l = torch.empty_like(none), torch.empty((0, 4), device="cuda")
    got = fa.paged_attention_forward(none, *g[:4], *dev, cu_q=_i32([0, 0, 0]), max_q=4, out=o, lse=l,
                                     stream=torch.cuda.Stream())
    assert got[0] is o and got[1] is l
    # no request at all
    out, lse = fa.paged_attention_forward(none, *g[:4], dev[0][:0], dev[1][:0])
    assert out.shape == (0, 4, d) and lse.shape == (0, 4)
    sel, count = fa.kv_page_select(none, g[4], g[2], dev[0][:0], dev[1][:0], 16, 3)
    assert sel.shape == (0, 2, 3) and count.shape == (0, 2)
    out, lse = fa.paged_attention_forward(none, *g[:4], dev[0][:0], dev[1][:0], selected=sel, selected_count=count)
    assert out.shape == (0, 4, d)
    # one query per request is still asked for where there are requests, and wrong tensors still refused
    with pytest.raises(fa.FaError):
        fa.paged_attention_forward(none, *g[:4], *dev)
    with pytest.raises(ValueError):
        fa.paged_attention_forward(none, *g[:4], *dev, cu_q=_i32([0, 0]))
    _ok()


# ------------------------------------------------- page numbers that cannot be
@pytest.mark.parametrize("P", [16, 64, 128])
@pytest.mark.parametrize("where", ["table", "stack", "given back"])
def test_tables_bad_page_numbers_give_no_slot(P, where):
    """A negative page, or one whose slots would pass 32 bits (and wrap to another page's): the tokens on it
    get no slot and the call is reported; the others have theirs."""
    fa = _fa()
    for page in (-1, -(1 << 31), (1 << 31) // P + 3, (1 << 31) - 1):
        # request 0 goes on inside the page it holds, request 1 needs pages, request 2 ends, request 3 is sound
        new, lens = np.array([2, 2 * P + 1, -1, 3]), np.array([5, 0, 4, 7])
        table = np.full((4, 4), -9)
        table[0, 0], table[2, 0], table[3, 0] = 11, 12, 13
        free = np.array([21, 22, 0, 0])
        if where == "table":
            table[0, 0] = page
        elif where == "stack":
            free[1] = page
        else:
            table[2, 0] = page
        T = 2 * P + 10
        want = ref.tables_step(new, lens, table, free, 2, P, T)
        assert want["status"] == 0
        got, g = base._step(new, lens, table, free, 2, P, T)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
        _ok()
        place = want["slots"] % P
        good = np.array([11, 22, 12, 13, 21])
        ok = np.isin(want["slots"] // P, good) & (want["slots"] >= 0)
        slots = got[0].cpu().numpy()
        np.testing.assert_array_equal(slots, np.where(ok, want["slots"], -1))
        assert (~ok[:int(want["cu"][-1])]).any() and ok.any() and (place[ok] == slots[ok] % P).all()
        np.testing.assert_array_equal(got[1].cpu().numpy(), want["cu"])
        np.testing.assert_array_equal(got[2].cpu().numpy(), want["lens"])
        with pytest.raises(fa.FaError):
            base._step(new, lens, table, free, 2, P, T, check=True)


def test_tables_largest_page_number():
    """The last page whose slots 32 bits hold."""
    for P in (16, 128):
        page = (1 << 31) // P - 1
        new, lens, table = np.array([P]), np.array([0]), np.full((1, 2), -1)
        want = ref.tables_step(new, lens, table, np.array([page]), 1, P, P)
        got, g = base._step(new, lens, table, np.array([page]), 1, P, P, check=True)
        base._check_step(got, g, want)
