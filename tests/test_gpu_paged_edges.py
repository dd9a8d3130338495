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


# ------------------------------------------------- slots left out of an append
def _append_sparse(cache, kv, slots, rows, dtype, bounds=True):
    """The tokens (kv, slots) at the given rows of a call whose other rows hold NaN and negative slots."""
    torch = _torch()
    T = int(rows[-1]) + 1 + 40
    x = torch.full((2, T, *kv.shape[2:]), float("nan"), dtype=kv.dtype)
    s = np.random.default_rng(len(rows)).choice([-1, -7, -(1 << 31)], size=T)
    x[:, rows], s[rows] = kv, slots
    g = base._append(cache, x, s, bounds=bounds)
    _ok()
    cache.append(*(y.double().numpy() for y in kv), slots, bounds=bounds)
    base._same_cache(g, cache, bounds)


@pytest.mark.parametrize("Hk,P,d,dtype", [(1, 16, 64, "bf16"), (3, 32, 96, "fp16"), (2, 128, 128, "bf16"), (1, 64, 256, "fp16")])
@pytest.mark.parametrize("drop", [0.05, 0.5, 0.9])
def test_append_with_rows_left_out_between_tokens(Hk, P, d, dtype, drop):
    """Rejected drafts, padded batches: rows without a slot anywhere, also between the tokens of one page."""
    pieces = [(0, 1), (P - 1, 1), (P - 1, 2), (3, 1), (0, P), (0, 3 * P + 5), (P, 7), (P + 5, P), (2 * P - 1, P + 2),
              (7, 3), (1, 5), (0, 9)]
    cache, kv, slots = base._append_case(Hk, P, d, pieces, dtype, 261 + d)
    rng = np.random.default_rng(261 + P)
    gaps = np.minimum(rng.geometric(1 - drop, size=len(slots)), 128)         # rows to the next token
    far = rng.random(len(slots)) < 0.03
    gaps[far] = rng.choice([127, 128], size=int(far.sum()))                  # the most there may be
    _append_sparse(cache, kv, slots, np.cumsum(gaps) - 1 + 5, dtype)


@pytest.mark.parametrize("T", [20, 700, 40000])
def test_append_rows_left_out_and_windows(T):
    """Runs of whole pages of 128 whose rows pass the 256 that a CTA looks at, beginnings behind rows left out,
    values that grow (a scale taken from part of a run would be too small), with few and many tokens."""
    rng = np.random.default_rng(T)
    P, pieces, n = 128, [], 0
    while n < T:
        k = int(rng.choice([1, 5, 127, 128, 129, 300]))
        pieces.append((int(rng.integers(0, P)) if rng.random() < 0.7 else 0, k))
        n += k
    cache, kv, slots = base._append_case(1, P, 16, pieces, "bf16", 271 + T)
    kv *= _torch().from_numpy(2.0 ** (np.arange(len(slots)) % 97 / 8.0))[None, :, None, None].to(kv.dtype)
    style = rng.random(len(slots))
    gaps = np.where(style < 0.8, 1, np.where(style < 0.95, rng.integers(2, 12, len(slots)), rng.integers(60, 129, len(slots))))
    _append_sparse(cache, kv, slots, np.cumsum(gaps) - 1, "bf16", bounds=T < 1000)


@pytest.mark.parametrize("L", [8, 64, 500])
def test_append_of_a_padded_batch(L):
    """[requests, L] rows, each request's tokens first (and once: last) in its L rows."""
    rng = np.random.default_rng(L)
    for first in (True, False):
        n = rng.integers(0, min(L, 150) + 1, 30)
        pieces = [(int(rng.integers(0, 200)), int(k)) for k in n if k]
        cache, kv, slots = base._append_case(2, 64, 64, pieces, "fp16", 281 + L)
        rows = np.concatenate([b * L + (0 if first else L - k) + np.arange(k) for b, k in enumerate(n)])
        _append_sparse(cache, kv, slots, rows, "fp16")


def test_append_slots_with_a_gap_are_reported_and_not_stored():
    """A page holds no gaps: tokens behind one are left out, those before it and other pages' are stored; with rows
    left out at the gap as well."""
    fa = _fa()
    for between in (0, 1, 127):
        for jump in (2, 5, 0, -1):
            cache, kv, slots = base._append_case(2, 32, 64, [(0, 20), (3, 1), (0, 9), (33, 4)], "bf16", 291)
            s, at = slots.copy(), 5
            s[at:20] += jump - 1                                             # row 5 is not the next place
            keep = np.ones(len(s), bool)
            keep[at:20] = False
            gap = np.ones(len(s), np.int64)
            gap[at] += between
            rows = np.cumsum(gap) - 1
            torch = _torch()
            x = torch.full((2, int(rows[-1]) + 1, *kv.shape[2:]), float("nan"), dtype=kv.dtype)
            y = np.full(int(rows[-1]) + 1, -1)
            x[:, rows], y[rows] = kv, s
            g = base._append(cache, x, y)
            assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG, (between, jump)
            _ok()
            cache.append(*(z.double().numpy() for z in kv[:, keep]), slots[keep])
            base._same_cache(g, cache)


# ------------------------------------------------- pending statuses
def test_a_status_of_each_kind_is_reported():
    """A wait that ran out in fa_fwd and bad data of a paged call, both pending: one answer after the other."""
    torch, fa = _torch(), _fa()
    B, H, N, d = 1, 1, 256, 64
    x = torch.randn((B, H, N, d), device="cuda").half()
    o, lse = torch.empty_like(x), torch.empty((B, H, N), device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    case = base._attend_case([40, 40], [1, 1], 1, 2, 16, 64, "fp16", 221)
    bad = case[1].copy()
    bad[1, 0] = -1
    for first in (0, 1):
        for step in (first, 1 - first):
            if step:
                assert fa.fa_fwd_debug(x.data_ptr(), x.data_ptr(), x.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                                       0.125, 0, fa.FA_FP16, s, 1, 0.05) == fa.FA_OK
            else:
                base._attend(case[0], bad, *case[2:], [1, 1])
        got = [fa.fa_check_device_status(s) for _ in range(3)]
        assert sorted(got[:2]) == sorted([fa.FA_ERR_TIMEOUT, fa.FA_ERR_INVALID_ARG]), got
        assert got[2] == fa.FA_OK


# ------------------------------------------------- bad device data on every kernel
@pytest.mark.parametrize("d", [64, 96, 128, 160, 256])
@pytest.mark.parametrize("splits", [1, 2])
def test_bad_pages_of_prompts_are_reported(d, splits):
    fa = _fa()
    news = [40, 30]
    cache, table, lens, cu, q = base._attend_case([100, 300], news, 1, 2, 16, d, "fp16", 231 + d)
    good = base._attend(cache, table, lens, cu, q, news, num_splits=splits)
    _ok()
    for at, entry in ((3, cache.pages), (0, -1), (18, 1 << 30), (7, -(1 << 31))):
        t = table.copy()
        t[1, at] = entry
        out, lse = base._attend(cache, t, lens, cu, q, news, num_splits=splits)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG, (at, entry)
        _ok()
        assert _torch().equal(out[:40], good[0][:40]) and _torch().equal(lse[:40], good[1][:40])


@pytest.mark.parametrize("splits", [1, 2, 3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_bad_selections_are_reported(d, splits):
    """Counts outside [0, keep] and indices outside the table: reported, the other request is served."""
    fa = _fa()
    case = base._select_case([900, 900], 2, 2, 16, d, "bf16", 241 + d)
    cache, table, lens, cu, q = case
    g, keep = cache.cuda(), 5
    sel = np.tile(np.array([1, 4, 9, 30, 56]), (2, 2, 1))
    count = np.full((2, 2), keep)

    def call(s, n):
        return fa.paged_attention_forward(q.cuda(), *g[:4], _i32(table), _i32(lens), selected=_i32(s),
                                          selected_count=_i32(n), num_splits=splits)

    good = call(sel, count)
    _ok()
    base._check_attend(case, *good, selected=[[list(r) for r in rows] for rows in sel])
    for what, value in (("count", keep + 1), ("count", -1), ("index", table.shape[1]), ("index", -1),
                        ("index", (1 << 31) - 1), ("index", -(1 << 31))):
        s, n = sel.copy(), count.copy()
        if what == "count":
            n[1, 1] = value
        else:
            s[1, 1, 2] = value
        out, lse = call(s, n)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG, (what, value)
        _ok()
        assert _torch().equal(out[0], good[0][0]) and _torch().equal(lse[0], good[1][0])


def test_bad_selections_of_equal_shares_are_reported():
    import ctypes
    torch, fa = _torch(), _fa()
    B, Hk, G, P, d = 36, 1, 4, 16, 128
    case = base._select_case([900] * B, Hk, G, P, d, "bf16", 251)
    cache, table, lens, cu, q = case
    g, keep = cache.cuda(), 64 * 30
    rng = np.random.default_rng(251)
    sel, count = np.full((B, Hk, keep), -1), np.full((B, Hk), 20)
    for b in range(B):
        sel[b, 0, :20] = np.sort(rng.choice(57, size=20, replace=False))

    def call(s, n):
        return fa.paged_attention_forward(q.cuda(), *g[:4], _i32(table), _i32(lens), selected=_i32(s), selected_count=_i32(n))

    a = fa.fa_paged_args()
    p = g[0].data_ptr()
    a.q = a.o = a.lse = a.block_table = a.lens = a.selected = a.selected_count = p
    a.cache = fa.fa_kv_cache(p, p, p, p, None, cache.pages, P, Hk, d)
    a.T, a.B, a.Hq, a.max_q, a.max_pages, a.num_selected = B, B, Hk * G, 1, table.shape[1], keep
    a.q_stride[:] = a.o_stride[:] = [Hk * G * d, d]
    a.scale, a.causal, a.dtype, a.num_splits = 0.1, 1, fa.FA_BF16, 0
    assert fa.library().fa_paged_num_splits(ctypes.addressof(a)) == 0      # (this is the way that is taken)
    good = call(sel, count)
    _ok()
    base._check_attend(case, *good, selected=[[list(r[r >= 0]) for r in rows] for rows in sel])
    others = np.arange(B) != 17
    for what, value in (("count", keep + 1), ("count", -1), ("index", table.shape[1]), ("index", -7)):
        s, n = sel.copy(), count.copy()
        if what == "count":
            n[17, 0] = value
        else:
            s[17, 0, 3] = value
        out, lse = call(s, n)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG, (what, value)
        _ok()
        keep_rows = torch.from_numpy(others).cuda()
        assert torch.equal(out[keep_rows], good[0][keep_rows]) and torch.equal(lse[keep_rows], good[1][keep_rows])
