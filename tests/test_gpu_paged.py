"""The operators around the paged 8-bit cache (include/fa_paged.h) on the GPU, against their
definitions in 64 bits or whole numbers (tests/paged_ref.py)."""
import math

import numpy as np
import pytest

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from online_softmax_tiling_gb300 import build
    build.build()
    yield


def _torch():
    import torch
    return torch


def _fa():
    import online_softmax_tiling_gb300 as fa
    return fa


def _dt(name):
    return {"bf16": _torch().bfloat16, "fp16": _torch().float16}[name]


def _i32(x):
    return _torch().as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _ok(stream=None):
    assert _fa().fa_check_device_status(stream) == _fa().FA_OK


# ------------------------------------------------------------------ tables
def _tables(B, P, top, seed, new=None, lens=None, spare=3, extra_cols=1):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top + 1, B) if lens is None else np.asarray(lens)
    if new is None:
        new = rng.integers(0, 3 * P, B)
        new[rng.random(B) < 0.2] = -1
        new[rng.random(B) < 0.2] = 0
    new = np.asarray(new)
    have = -(-lens // P)
    want = -(-np.where(new < 0, 0, lens + np.maximum(new, 0)) // P)
    M = int(max(have.max(), want.max())) + extra_cols
    need = np.where(new < 0, 0, want - have).sum()
    total = int(have.sum() + need) + spare
    perm = rng.permutation(total)
    table = np.full((B, M), -7)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = np.full(total, -9)
    free[:total - at] = perm[at:]
    return new, lens, table, free, total - at


def _step(new, lens, table, free, count, P, max_tokens, **kw):
    g = [_i32(new), _i32(lens), _i32(table), _i32(free), _i32([count])]
    before = [x.clone() for x in g]
    out = _fa().kv_tables_step(*g, page_size=P, max_tokens=max_tokens, **kw)
    assert all(_torch().equal(g[i], before[i]) for i in (0, 1, 4))   # inputs stay as they were
    return out, g


def _check_step(got, g, want):
    slots, cu, lens, count, status = (x.cpu().numpy() for x in got)
    assert status[0] == want["status"]
    np.testing.assert_array_equal(cu, want["cu"])
    np.testing.assert_array_equal(slots, want["slots"])
    np.testing.assert_array_equal(lens, want["lens"])
    assert count[0] == want["count"]
    np.testing.assert_array_equal(g[2].cpu().numpy(), want["table"])
    np.testing.assert_array_equal(g[3].cpu().numpy(), want["free"])


@pytest.mark.parametrize("B,P,top,seed", [
    (1, 16, 0, 1), (1, 128, 300, 2), (2, 64, 64, 3), (7, 32, 200, 4), (33, 16, 1000, 5),
    (512, 64, 90, 6), (513, 16, 40, 7), (1537, 16, 30, 8)])
@pytest.mark.parametrize("room", [0, 5])
def test_tables_step(B, P, top, seed, room):
    new, lens, table, free, count = _tables(B, P, top, seed)
    T = int(np.maximum(new, 0).sum()) + room
    want = ref.tables_step(new, lens, table, free, count, P, T)
    got, g = _step(new, lens, table, free, count, P, T, check=True)
    _check_step(got, g, want)
    # the same step again, from the same inputs: the same result
    again = _fa().kv_tables_step(*g, page_size=P, max_tokens=T)
    _check_step(again, g, want)


def test_tables_largest_batch():
    B, P = 16384, 16
    new, lens, table, free, count = _tables(B, P, 40, 11, new=np.ones(B, np.int64))
    want = ref.tables_step(new, lens, table, free, count, P, B)
    _check_step(*_step(new, lens, table, free, count, P, B), want)
    with pytest.raises(_fa().FaError):
        _step(np.ones(B + 1), np.ones(B + 1), np.zeros((B + 1, 2)), free, count, P, B + 1)


def test_tables_lengths_at_page_borders():
    P = 32
    lens = [0, 0, 1, P - 1, P, P + 1, 2 * P, 5, 0, P]
    new = [0, 1, P - 1, 1, 1, P - 1, 0, -1, -1, -1]
    new, lens, table, free, count = _tables(10, P, 0, 12, new=new, lens=lens)
    want = ref.tables_step(new, lens, table, free, count, P, 70)
    _check_step(*_step(new, lens, table, free, count, P, 70), want)


def test_tables_pages_given_back_are_taken_in_the_same_step():
    P = 16
    new, lens, table, free, _ = _tables(3, P, 0, 13, new=[-1, 60, -1], lens=[50, 0, 20], spare=0)
    table[0, :4], table[2, :2] = [3, 1, 4, 5], [9, 2]
    free[:] = -9
    want = ref.tables_step(new, lens, table, free, 0, P, 60)
    assert want["status"] == 0 and set(want["table"][1, :4]) == {2, 9, 5, 4}
    _check_step(*_step(new, lens, table, free, 0, P, 60), want)


@pytest.mark.parametrize("what", ["pages", "tokens", "row", "length", "stack", "count"])
def test_tables_refused_steps_change_nothing(what):
    P = 16
    new, lens, table, free, count = _tables(20, P, 100, 14)
    T = int(np.maximum(new, 0).sum())
    code = 1
    if what == "pages":
        need = count - 3
        new, lens = new.copy(), lens.copy()
        new[new < 0] = 0
        count, code = max(0, need - 1), 6
    elif what == "tokens":
        T -= 1
    elif what == "row":
        new = new.copy()
        new[4] = table.shape[1] * P + 1 - lens[4]
        T += new[4]
    elif what == "length":
        lens = lens.copy()
        lens[7] = -1
    elif what == "stack":
        free = free[:count]
        if not (new < 0).any():
            new[0] = -1
    else:
        count = -1
    want = ref.tables_step(new, lens, table, free, count, P, T)
    assert want["status"] == code
    got, g = _step(new, lens, table, free, count, P, T)
    _check_step(got, g, want)
    with pytest.raises(_fa().FaError):
        _step(new, lens, table, free, count, P, T, check=True)


def test_tables_many_steps_keep_every_page_once():
    """A server's life: steps from one another's outputs; no page is ever lost or held twice."""
    rng = np.random.default_rng(15)
    P, B, M, total = 16, 24, 12, 150
    lens, table = np.zeros(B, np.int64), np.full((B, M), -1)
    g_table, g_free = _i32(table), _i32(rng.permutation(total))
    g_lens, g_count = _i32(lens), _i32([total])
    free, count = g_free.cpu().numpy().astype(np.int64), total
    for step in range(40):
        new = rng.integers(0, 40, B)
        new[rng.random(B) < 0.3] = -1
        new = np.where(lens + new > M * P, -1, new)
        T = 1000
        want = ref.tables_step(new, lens, table, free, count, P, T)
        slots, cu, g_lens, g_count, status = _fa().kv_tables_step(_i32(new), g_lens, g_table, g_free, g_count, P, T)
        assert status.item() == want["status"]
        np.testing.assert_array_equal(slots.cpu().numpy(), want["slots"])
        lens, table, free, count = want["lens"], want["table"], want["free"], int(want["count"])
        np.testing.assert_array_equal(g_table.cpu().numpy(), table)
        held = np.concatenate([table[b, :-(-lens[b] // P)] for b in range(B)] + [free[:count]])
        assert sorted(held) == list(range(total))


# ------------------------------------------------------------------ append
def _append_case(Hk, P, d, pieces, dtype, seed, pages=None):
    """pieces: (page list start handled by a random table) [(tokens before, new tokens)]."""
    rng = np.random.default_rng(seed)
    need = sum(-(-(a + n) // P) for a, n in pieces)
    pages = need + 3 if pages is None else pages
    cache = ref.Cache(pages, Hk, P, d, seed)
    perm, at, slots = rng.permutation(pages), 0, []
    for a, n in pieces:
        k = -(-(a + n) // P)
        row = perm[at:at + k]
        at += k
        pos = np.arange(a, a + n)
        slots += list(row[pos // P] * P + pos % P)
        if a % P:
            cache.set_bounds(row[a // P], a % P)
    T = len(slots)
    torch = _torch()
    kv = rng.standard_normal((2, T, Hk, d)) * np.exp(rng.standard_normal((2, T, Hk, 1)))
    kv = torch.from_numpy(kv).to(_dt(dtype))
    return cache, kv, np.array(slots)


def _append(cache, kv, slots, bounds=True, **kw):
    g = cache.cuda()
    _fa().kv_cache_append(kv[0].cuda(), kv[1].cuda(), _i32(slots), *g[:4], k_bounds=g[4] if bounds else None, **kw)
    return g


def _same_cache(g, cache, bounds=True):
    torch = _torch()
    for i, n in enumerate("kv"):
        np.testing.assert_array_equal(g[2 + i].cpu().numpy(), cache.scale[n].astype(np.float32))
        got = g[i].view(torch.uint8).cpu().numpy()
        nan = np.isnan(ref.VALUES[cache.codes[n]])
        np.testing.assert_array_equal(np.where(nan, 127, got & np.where(nan, 127, 255)),
                                      np.where(nan, 127, cache.codes[n]))
    if bounds:
        np.testing.assert_array_equal(g[4].cpu().numpy(), cache.bounds)


@pytest.mark.parametrize("Hk,P,d", [(1, 16, 16), (2, 16, 64), (3, 32, 80), (2, 64, 96), (1, 128, 128),
                                    (2, 64, 128), (1, 32, 192), (1, 128, 256), (5, 16, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append(Hk, P, d, dtype):
    """Pieces that begin and end anywhere in pages, from one token to several pages."""
    pieces = [(0, 1), (P - 1, 1), (P - 1, 2), (3, 1), (0, P), (0, 3 * P + 5), (P, 7), (P + 5, P), (2 * P - 1, P + 2)]
    cache, kv, slots = _append_case(Hk, P, d, pieces, dtype, 21 + d)
    g = _append(cache, kv, slots)
    _ok()
    cache.append(*(x.double().numpy() for x in kv), slots)
    _same_cache(g, cache)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 300])
def test_append_single_tokens(T):
    """A decode step: every token another page; and without bounds."""
    cache, kv, slots = _append_case(4, 16, 128, [(i % 40, 1) for i in range(T)], "bf16", 22)
    g = _append(cache, kv, slots, bounds=False)
    before = cache.bounds.copy()
    cache.append(*(x.double().numpy() for x in kv), slots, bounds=False)
    _same_cache(g, cache)
    np.testing.assert_array_equal(g[4].cpu().numpy(), before)


def test_append_many_tokens_use_the_wide_chunks():
    cache, kv, slots = _append_case(8, 64, 64, [(5, 1500), (0, 700), (64, 1), (1, 1)], "fp16", 23)
    g = _append(cache, kv, slots)
    cache.append(*(x.double().numpy() for x in kv), slots)
    _same_cache(g, cache)


def test_append_skips_negative_slots_and_leaves_other_pages():
    cache, kv, slots = _append_case(2, 16, 64, [(0, 40), (10, 20)], "bf16", 24)
    slots[::3] = -1
    kv[:, ::3] = float("nan")
    # (a gap in a page breaks its run; the next one would be a second run of the same page)
    slots[1:] = np.where(slots[1:] // 16 == np.roll(slots, 1)[1:] // 16, slots[1:], -1)
    keep, seen = [], set()
    for s in slots:
        if s >= 0 and s // 16 not in seen:
            seen.add(s // 16)
            keep.append(s)
        else:
            keep.append(-1)
    slots = np.array(keep)
    g = _append(cache, kv, slots)
    _ok()
    cache.append(*(x.double().numpy() for x in kv), slots)
    _same_cache(g, cache)


def test_append_special_values():
    """Zeros, infinities, NaN, the smallest and largest numbers; a page of each kind, fresh and appended to."""
    torch = _torch()
    inf, nan = math.inf, math.nan
    for dtype in ("bf16", "fp16"):
        f = torch.finfo(_dt(dtype))
        rows = [0.0, -0.0, inf, -inf, nan, f.max, f.tiny, f.smallest_normal * f.eps, 448.0, 449.0, 2.0 ** -9, 240.0 * 2 ** -20]
        cache, kv, slots = _append_case(1, 16, 64, [(0, 16)] * len(rows) + [(5, 3)] * len(rows), dtype, 25)
        for i, r in enumerate(rows):
            kv[:, 16 * i:16 * i + 16] *= 0.01
            kv[:, 16 * i + 3, 0, 5] = r
            at = 16 * len(rows) + 3 * i
            kv[:, at:at + 3] = r
        g = _append(cache, kv, slots)
        _ok()
        cache.append(*(x.double().numpy() for x in kv), slots)
        _same_cache(g, cache)


def test_append_growing_scale_rounds_older_codes():
    """Token by token with ever larger values: the scale grows and older codes are rounded again."""
    P, d = 32, 64
    cache = ref.Cache(2, 2, P, d, 26, random=False)
    torch = _torch()
    rng = np.random.default_rng(26)
    x = torch.from_numpy(rng.standard_normal((2, P, 2, d)) * 2.0 ** np.linspace(-12, 12, P)[None, :, None, None]).bfloat16()
    g = cache.cuda()
    for t in range(P):
        _fa().kv_cache_append(x[0, t:t + 1].cuda(), x[1, t:t + 1].cuda(), _i32([P + t]), *g[:4], k_bounds=g[4])
        cache.append(x[0, t:t + 1].double().numpy(), x[1, t:t + 1].double().numpy(), np.array([P + t]))
    _ok()
    _same_cache(g, cache)
    # and a page that is used again starts anew, however large its old scale was
    y = x[:, :2] * 2.0 ** -10
    _fa().kv_cache_append(y[0].cuda(), y[1].cuda(), _i32([P, P + 1]), *g[:4], k_bounds=g[4])
    cache.append(y[0].double().numpy(), y[1].double().numpy(), np.array([P, P + 1]))
    _same_cache(g, cache)


def test_append_strided_and_other_stream():
    torch = _torch()
    cache, kv, slots = _append_case(3, 32, 128, [(3, 50), (0, 33)], "fp16", 27)
    T = len(slots)
    wide = torch.zeros((T, 2, 5, 128), dtype=torch.float16, device="cuda")     # [T, k or v, head, d], padded heads
    wide[:, 0, 1:4], wide[:, 1, 1:4] = kv[0].cuda(), kv[1].cuda()
    g = cache.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _fa().kv_cache_append(wide[:, 0, 1:4], wide[:, 1, 1:4], _i32(slots), *g[:4], k_bounds=g[4], stream=s, check=True)
    torch.cuda.synchronize()
    cache.append(*(x.double().numpy() for x in kv), slots)
    _same_cache(g, cache)


def test_append_bad_slots_are_reported_and_not_stored():
    fa = _fa()
    cache, kv, slots = _append_case(2, 16, 64, [(0, 20), (16, 5)], "bf16", 28)
    bad = slots.copy()
    bad[20:] = cache.pages * 16 + np.arange(5)                # no such page
    g = _append(cache, kv, bad)
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
    _ok()
    good = np.where(np.arange(25) < 20, slots, -1)
    c2, kv2, _ = _append_case(2, 16, 64, [(0, 20), (16, 5)], "bf16", 28)
    c2.append(*(x.double().numpy() for x in kv2), good)
    _same_cache(g, c2)
    twice = slots.copy()
    twice[1] = slots[0]                                       # the same slot twice
    _append(cache, kv, twice)
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
    _ok()


# --------------------------------------------------------------- attention
def _attend_case(lens, news, Hk, G, P, d, dtype, seed):
    rng = np.random.default_rng(seed)
    lens, news = np.asarray(lens), np.asarray(news)
    need = -(-lens // P)
    pages = int(need.sum()) + 3
    cache = ref.Cache(pages, Hk, P, d, seed)
    M = max(1, int(need.max()))
    # entries behind a request's pages are never read: they may be anything
    table = rng.choice([-1, 1 << 30, -(1 << 31), 10 ** 6], size=(len(lens), M))
    perm, at = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        if lens[b] % P:  # what an earlier request left behind the last token: NaN, the largest code
            tail = cache.codes["k"][table[b, n - 1]][:, lens[b] % P:], cache.codes["v"][table[b, n - 1]][:, lens[b] % P:]
            for x in tail:
                x[...] = rng.choice([0x7F, 0xFF, 0x7E, 0xFE], size=x.shape)
    cu = np.concatenate([[0], np.cumsum(news)])
    q = _torch().from_numpy(rng.standard_normal((int(cu[-1]), Hk * G, d))).to(_dt(dtype))
    return cache, table, lens, cu, q


def _attend(cache, table, lens, cu, q, news, **kw):
    g = cache.cuda()
    force = kw.pop("force_cu", False)
    one = (np.diff(cu) == 1).all() and not force
    return _fa().paged_attention_forward(q.cuda(), *g[:4], _i32(table), _i32(lens), cu_q=None if one else _i32(cu),
                                         max_q=1 if one else max(1, int(np.max(news))), **kw)


def _check_attend(case, out, lse, causal=True, scale=None, selected=None, rows=slice(None)):
    cache, table, lens, cu, q = case
    d = q.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    r = ref.attend(cache, q.double().numpy(), table, lens, cu, scale, causal, selected)
    ref.check(out, lse, r, d, int(max(lens)), 448 * cache.scale["v"].max(), q.dtype, rows)


DECODE = [  # Hk, G, P, d
    (1, 1, 16, 64), (2, 4, 64, 128), (1, 8, 32, 256), (3, 2, 128, 96), (2, 5, 16, 80), (1, 16, 64, 128),
    (1, 24, 32, 64), (2, 3, 64, 16), (1, 2, 16, 192), (1, 40, 16, 128), (1, 17, 128, 256), (1, 96, 32, 128), (2, 71, 64, 64)]


@pytest.mark.parametrize("Hk,G,P,d", DECODE)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("splits", [0, 1, 2, 3, 16])
def test_decode(Hk, G, P, d, dtype, splits):
    """One query per request; lengths 0, 1, around tile and page borders, ragged ones."""
    lens = [0, 1, 15, 16, 17, P - 1, P, P + 1, 127, 300, 777]
    case = _attend_case(lens, [1] * len(lens), Hk, G, P, d, dtype, 31 + d + G)
    out, lse = _attend(*case, [1], num_splits=splits)
    _ok()
    _check_attend(case, out, lse)


@pytest.mark.parametrize("splits", [0, 1, 2, 4, 7, 8, 16, 64])
def test_decode_long(splits):
    """More than 32 chunks per warp (the lookups are refilled), and splits that stay empty."""
    case = _attend_case([9000, 40], [1, 1], 1, 4, 16, 128, "bf16", 41)
    out, lse = _attend(*case, [1, 1], num_splits=splits)
    _ok()
    _check_attend(case, out, lse)


PROMPT = [  # lens, news, Hk, G, P, d
    ([5, 40, 0, 300], [5, 3, 0, 17], 2, 4, 16, 128),
    ([33, 64, 200], [33, 1, 130], 1, 2, 32, 64),
    ([100, 7], [90, 7], 1, 3, 64, 256),
    ([1, 70, 129], [1, 66, 128], 2, 1, 16, 96),
    ([600, 500], [260, 300], 1, 8, 64, 128),
    ([300, 80], [200, 80], 2, 5, 128, 80),
]


@pytest.mark.parametrize("lens,news,Hk,G,P,d", PROMPT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,splits", [("bf16", 0), ("fp16", 1), ("bf16", 3)])
def test_several_queries(lens, news, Hk, G, P, d, causal, dtype, splits):
    case = _attend_case(lens, news, Hk, G, P, d, dtype, 51 + d + len(lens))
    out, lse = _attend(*case, news, causal=causal, num_splits=splits)
    _ok()
    _check_attend(case, out, lse, causal)


WIDE_PROMPT = [  # lens, news, Hk, G, P, d
    ([5, 40, 0, 300], [5, 25, 0, 17], 2, 4, 16, 256),
    ([33, 64, 200], [33, 20, 130], 1, 2, 32, 144),
    ([1, 63, 64, 65], [1, 63, 64, 65], 1, 1, 16, 192),
    ([128, 129, 2000], [128, 129, 37], 1, 3, 128, 160),
    ([700, 500], [260, 300], 1, 8, 64, 256),
    ([1300, 80], [200, 80], 2, 5, 128, 208),
]


@pytest.mark.parametrize("lens,news,Hk,G,P,d", WIDE_PROMPT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,splits", [("bf16", 0), ("fp16", 1), ("bf16", 3)])
def test_several_queries_of_wide_heads(lens, news, Hk, G, P, d, causal, dtype, splits):
    """Tiles of 64 keys and 128 packed rows: more tiles than stages, odd and even counts, ragged ends."""
    case = _attend_case(lens, news, Hk, G, P, d, dtype, 151 + d + len(lens))
    out, lse = _attend(*case, news, causal=causal, num_splits=splits)
    _ok()
    _check_attend(case, out, lse, causal)


@pytest.mark.parametrize("d", [128, 256])
def test_several_queries_over_a_wide_range_of_scales(d):
    """The running reference moves late and by much; rows of very different size; some see no key."""
    news = [100, 70]
    case = _attend_case([900, 30], news, 2, 2, 16, d, "bf16", 164 + d)
    cache, table, lens, cu, q = case
    rng = np.random.default_rng(64)
    cache.scale["v"] = 2.0 ** rng.integers(-30, 20, cache.scale["v"].shape)
    cache.scale["k"] = 2.0 ** rng.integers(-12, -3, cache.scale["k"].shape)
    q[3, 1] *= 50.0
    q[4, 0] *= 1e-20
    q[5, 2] = 0
    for splits in (1, 3):
        out, lse = _attend(*case, news, num_splits=splits)
        _ok()
        O, L, A, D = ref.attend(cache, q.double().numpy(), table, lens, cu, 1 / math.sqrt(d), True)
        ref.check(out, lse, (O, L, A, D), d, 900, 448 * cache.scale["v"].max(), q.dtype)
        assert (lse[100:140].isinf()).all() and (out[100:140] == 0).all()


def test_bad_pages_of_wide_heads_are_reported():
    fa = _fa()
    news = [40, 30]
    cache, table, lens, cu, q = _attend_case([100, 100], news, 1, 2, 16, 256, "fp16", 167)
    good = _attend(cache, table, lens, cu, q, news)
    _ok()
    for entry in (cache.pages, -1):
        t = table.copy()
        t[1, 3] = entry
        out, lse = _attend(cache, t, lens, cu, q, news)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
        _ok()
        assert _torch().equal(out[:40], good[0][:40])


@pytest.mark.parametrize("Hk,G,P,d", [(2, 4, 64, 128), (2, 1, 16, 64), (3, 16, 32, 96), (2, 5, 64, 256), (2, 20, 128, 128)])
@pytest.mark.parametrize("dtype,causal", [("bf16", True), ("fp16", False)])
def test_prompts_beside_single_tokens(Hk, G, P, d, dtype, causal):
    """One call of prompts, drafts, single tokens, requests without queries and without keys."""
    lens = [1, 300, 33, 700, 1, 64, 0, 500, 17, 40, 900, 128]
    news = [1, 1, 2, 300, 1, 0, 1, 8, 1, 40, 1, 3]
    case = _attend_case(lens, news, Hk, G, P, d, dtype, 171 + d + G)
    out, lse = _attend(*case, news, causal=causal)
    _ok()
    _check_attend(case, out, lse, causal)
    # the same call captured, and rows behind the last query left alone
    torch = _torch()
    cache, table, lens_, cu, q = case
    g, dev = cache.cuda(), (_i32(table), _i32(lens_), _i32(cu))
    pad = torch.cat([q, q[:4]]).cuda()
    o, l = torch.full_like(pad, 7.0), torch.full((pad.shape[0], Hk * G), 7.0, device="cuda")
    call = lambda: _fa().paged_attention_forward(pad, *g[:4], dev[0], dev[1], cu_q=dev[2], max_q=300, causal=causal, out=o, lse=l)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    o.fill_(7.0), l.fill_(7.0)
    graph.replay()
    _ok()
    assert torch.equal(o[:-4], out) and torch.equal(l[:-4], lse)
    assert (o[-4:] == 7).all() and (l[-4:] == 7).all()


@pytest.mark.parametrize("d", [64, 256])
def test_prompts_among_more_requests_than_threads(d):
    """1500 requests: a thread counts the row blocks of several."""
    rng = np.random.default_rng(180 + d)
    news = np.ones(1500, int)
    news[rng.choice(1500, 200, replace=False)] = 0
    news[[0, 1, 2, 640, 641, 900, 1498, 1499]] = [70, 3, 200, 9, 64, 130, 33, 65]
    lens = np.maximum(news, rng.integers(0, 40, 1500))
    lens[[2, 900]] += 300
    case = _attend_case(lens, news, 1, 4, 16, d, "bf16", 181)
    out, lse = _attend(*case, news)
    _ok()
    _check_attend(case, out, lse)


def test_queries_that_see_no_key():
    """More queries than keys: the first ones see nothing and get 0 and -inf."""
    news = [20, 140, 3]
    case = _attend_case([5, 30, 0], news, 1, 4, 16, 64, "fp16", 61)
    for splits in (1, 2):
        out, lse = _attend(*case, news, num_splits=splits)
        _ok()
        _check_attend(case, out, lse)
        assert (lse[:15].isinf()).all() and (out[:15] == 0).all()


def test_rows_behind_the_last_query_are_left():
    torch = _torch()
    news = [3, 5]
    cache, table, lens, cu, q = _attend_case([50, 70], news, 2, 2, 16, 128, "bf16", 62)
    pad = torch.cat([q, torch.full((4, 4, 128), float("nan"), dtype=q.dtype)])
    for splits in (1, 4, 5):
        out = torch.full_like(pad, 7.0, device="cuda")
        lse = torch.full((12, 4), 7.0, device="cuda")
        _attend(cache, table, lens, cu, pad, news, out=out, lse=lse, num_splits=splits)
        _ok()
        assert (out[8:] == 7).all() and (lse[8:] == 7).all()
        _check_attend((cache, table, lens, cu, q), out[:8], lse[:8])


def test_strided_queries_and_outputs():
    torch = _torch()
    case = _attend_case([90, 33, 200], [1, 1, 1], 2, 4, 32, 128, "fp16", 63)
    cache, table, lens, cu, q = case
    wide = torch.zeros((3, 8, 3, 128), dtype=q.dtype, device="cuda")    # q, k, v side by side per head
    wide[:, :, 1] = q.cuda()
    store = torch.full((8, 3, 136), 5.0, dtype=q.dtype, device="cuda")  # heads outermost, padded rows
    out = store.permute(1, 0, 2)[:, :, :128]
    g = cache.cuda()
    for splits in (1, 3):
        o, lse = _fa().paged_attention_forward(wide[:, :, 1], *g[:4], _i32(table), _i32(lens), out=out, num_splits=splits)
        _ok()
        assert o is out and (store[:, :, 128:] == 5).all()
        _check_attend(case, out, lse)


def test_wide_range_of_scales():
    """Keys and values whose pages differ by many powers of two."""
    case = _attend_case([400, 260], [1, 1], 2, 4, 16, 128, "bf16", 64)
    cache = case[0]
    rng = np.random.default_rng(64)
    cache.scale["v"] = 2.0 ** rng.integers(-30, 20, cache.scale["v"].shape)
    cache.scale["k"] = 2.0 ** rng.integers(-12, -3, cache.scale["k"].shape)
    for splits in (1, 3):
        out, lse = _attend(*case, [1, 1], num_splits=splits)
        _ok()
        cache_, table, lens, cu, q = case
        O, L, A, D = ref.attend(cache, q.double().numpy(), table, lens, cu, 1 / math.sqrt(128), True)
        ref.check(out, lse, (O, L, A, D), 128, 400, 448 * cache.scale["v"].max(), q.dtype)


def test_large_and_small_queries():
    """Query rows of very different size, one of zeros among them, and a large scale."""
    case = _attend_case([300, 20, 77], [1, 1, 1], 1, 4, 32, 64, "bf16", 65)
    q = case[4]
    q[0, 0] *= 100.0
    q[0, 1] *= 1e-20
    q[1, 2] = 0
    q[2, 3] *= 30.0
    out, lse = _attend(*case, [1, 1, 1], scale=0.3)
    _ok()
    _check_attend(case, out, lse, scale=0.3)


def test_offsets_beyond_32_bits():
    """Pages far beyond 2^31 bytes of codes."""
    torch = _torch()
    Hk, P, d = 4, 128, 256
    pages = (1 << 31) // (Hk * P * d) + 40
    small = ref.Cache(5, Hk, P, d, 66)
    g = small.cuda()
    far = [pages - 1, 0, pages - 17, pages // 2, pages - 3]
    big = [torch.zeros((pages, Hk, P, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.ones((pages, Hk), dtype=torch.float32, device="cuda") for _ in range(2)]
    for i in range(2):
        big[i][far] = g[i].view(torch.uint8)
        sc[i][far] = g[2 + i]
    rng = np.random.default_rng(66)
    q = torch.from_numpy(rng.standard_normal((1, 8, d))).bfloat16()
    kc, vc = (x.view(torch.float8_e4m3fn) for x in big)
    lens = [5 * P - 3]
    out, lse = _fa().paged_attention_forward(q.cuda(), kc, vc, *sc, _i32([far]), _i32(lens))
    _ok()
    _check_attend((small, np.arange(5)[None], lens, [0, 1], q), out, lse)
    # and an append into the last page
    kv = torch.from_numpy(rng.standard_normal((2, 3, Hk, d))).bfloat16()
    slots = (pages - 1) * P + np.arange(P - 3, P)
    _fa().kv_cache_append(kv[0].cuda(), kv[1].cuda(), _i32(slots), kc, vc, *sc)
    _ok()
    small.append(*(x.double().numpy() for x in kv), np.arange(P - 3, P), bounds=False)
    for i, n in enumerate("kv"):
        np.testing.assert_array_equal(big[i][far].cpu().numpy(), small.codes[n])


def test_bad_device_data_is_reported():
    """Lengths, pages and row marks that cannot be are caught by the kernels' own checks."""
    fa = _fa()
    case = _attend_case([100, 100], [1, 1], 1, 2, 16, 64, "fp16", 67)
    cache, table, lens, cu, q = case
    good = _attend(*case, [1, 1])
    _ok()
    for change in ("page", "negative page", "length", "negative length", "marks"):
        t, l, c, kw = table.copy(), lens.copy(), cu.copy(), {}
        if change == "page":
            t[1, 3] = cache.pages
        elif change == "negative page":
            t[1, 0] = -1
        elif change == "length":
            l[1] = table.shape[1] * 16 + 1
        elif change == "negative length":
            l[1] = -5
        else:
            c[2], kw = 900, dict(force_cu=True)
        out, lse = _attend(cache, t, l, c, q, [1, 1], **kw)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG, change
        _ok()
        assert _torch().equal(out[0], good[0][0])              # the other request is served


def _wide_table(table, P, keys):
    """The same requests with a table that has room for `keys` keys (which decides how the work is split)."""
    wide = np.full((table.shape[0], -(-keys // P)), -5)
    wide[:, :table.shape[1]] = table
    return wide


EVEN = [  # lens, news, Hk, G, P, d
    ([0, 900, 1, 64, 333, 0, 0, 700, 31, 32, 33, 512, 5, 128, 640, 2], 1, 2, 4, 16, 128),
    ([100 + 37 * i for i in range(20)], 1, 2, 8, 64, 64),
    ([600 - 30 * i for i in range(20)], 1, 2, 7, 32, 256),
    ([40 * i for i in range(16)], [2, 0, 1, 2] * 4, 2, 4, 128, 128),
    ([3000, 1, 2900, 0] * 8, 1, 1, 16, 16, 96),
    ([250 + i for i in range(30)], [3, 1, 0, 2, 3] * 6, 1, 10, 64, 80),
    ([777, 3, 500] * 8, 1, 2, 24, 16, 64),
    ([90, 0, 45] * 10, 1, 1, 12, 16, 192)]


@pytest.mark.parametrize("lens,news,Hk,G,P,d", EVEN)
@pytest.mark.parametrize("causal", [True, False])
def test_even_shares(lens, news, Hk, G, P, d, causal):
    """All requests' keys dealt out in equal shares: units cut into many parts, whole ones between them,
    requests without keys or without queries."""
    torch, fa = _torch(), _fa()
    news = [news] * len(lens) if isinstance(news, int) else [min(n, max(m, 1)) for n, m in zip(news, lens)]
    case = _attend_case(lens, news, Hk, G, P, d, "bf16" if d % 32 else "fp16", 101 + d + G)
    cache, table, lens, cu, q = case
    keys = 456 * 66 * 32 // (len(lens) * Hk)
    wide = _wide_table(table, P, keys)
    a = fa.fa_paged_args()
    one = (np.diff(cu) == 1).all()
    pad = torch.cat([q, q[:2]]) if not one else q
    out = torch.full_like(pad, 3.0, device="cuda")
    lse = torch.full(pad.shape[:2], 3.0, device="cuda")
    a.q, a.o, a.lse, a.block_table, a.lens = out.data_ptr(), out.data_ptr(), lse.data_ptr(), lse.data_ptr(), lse.data_ptr()
    a.cu_q = None if one else lse.data_ptr()
    a.cache = fa.fa_kv_cache(out.data_ptr(), out.data_ptr(), lse.data_ptr(), lse.data_ptr(), None, cache.pages, P, Hk, d)
    a.T, a.B, a.Hq, a.max_q, a.max_pages = pad.shape[0], len(lens), Hk * G, 1 if one else int(max(news)), wide.shape[1]
    a.q_stride[:] = a.o_stride[:] = [Hk * G * d, d]
    a.scale, a.causal, a.dtype, a.num_splits = 0.1, causal, fa.FA_BF16, 0
    import ctypes
    assert fa.library().fa_paged_num_splits(ctypes.addressof(a)) == 0      # (this is the way that is taken)
    for _ in range(2):
        _attend(cache, wide, lens, cu, pad, news, causal=causal, out=out, lse=lse)
        _ok()
        _check_attend(case, out[:len(q)], lse[:len(q)], causal)
        assert (out[len(q):] == 3).all() and (lse[len(q):] == 3).all()


def test_even_shares_in_a_graph_follow_the_lengths():
    """A captured call reads lengths, tables and queries when it is replayed."""
    torch, fa = _torch(), _fa()
    case = _attend_case([500 + 11 * i for i in range(40)], [1] * 40, 1, 4, 16, 128, "fp16", 103)
    cache, table, lens, cu, q = case
    wide, g = _i32(_wide_table(table, 16, 456 * 66 * 32 // 40)), cache.cuda()
    d_lens, d_q = _i32(lens), q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.paged_attention_forward(d_q, *g[:4], wide, d_lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fa.paged_attention_forward(d_q, *g[:4], wide, d_lens)
    rng = np.random.default_rng(103)
    for _ in range(4):
        now = np.where(rng.random(40) < 0.2, 0, rng.integers(1, lens + 1))
        q2 = torch.from_numpy(rng.standard_normal(q.shape)).half()
        d_lens.copy_(_i32(now))
        d_q.copy_(q2)
        graph.replay()
        _ok()
        _check_attend((cache, table, now, cu, q2), out, lse)


def test_even_shares_of_selected_pages():
    lens = [0, 5000, 64, 3000, 17, 900] * 6
    case = _select_case(lens, 1, 4, 16, 128, "bf16", 102)
    cache, table, lens, cu, q = case
    keep = 64 * 30                                            # (room for them decides how the work is split)
    g = cache.cuda()
    rng = np.random.default_rng(102)
    sel = np.full((len(lens), 1, keep), -1)
    count = np.zeros((len(lens), 1), np.int64)
    for b, n in enumerate(lens):
        pages = -(-n // 16)
        pick = np.sort(rng.choice(pages, size=min(pages, 40 + b), replace=False)) if pages else []
        sel[b, 0, :len(pick)], count[b] = pick, len(pick)
    out, lse = _fa().paged_attention_forward(q.cuda(), *g[:4], _i32(table), _i32(lens), selected=_i32(sel),
                                             selected_count=_i32(count))
    _ok()
    _check_attend(case, out, lse, selected=[[list(r[r >= 0]) for r in rows] for rows in sel])


# --------------------------------------------------------- page selection
def _select_case(lens, Hk, G, P, d, dtype, seed):
    case = _attend_case(lens, [1] * len(lens), Hk, G, P, d, dtype, seed)
    cache, table = case[0], case[1]
    for b, n in enumerate(lens):
        for j in range(-(-n // P)):
            cache.set_bounds(table[b, j], min(P, n - j * P))
    return case


@pytest.mark.parametrize("lens,Hk,G,P,d,keep", [
    ([0, 1, 16, 17, 400, 2000], 2, 4, 16, 128, 5), ([700, 3000], 3, 1, 32, 64, 1), ([5000], 1, 8, 16, 256, 64),
    ([1000, 999, 64], 2, 5, 64, 96, 3), ([9000, 12], 1, 2, 16, 80, 200), ([640], 1, 4, 128, 16, 4),
    ([640], 1, 4, 64, 64, 10), ([640], 1, 4, 64, 64, 30), ([900, 70], 1, 70, 16, 128, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_select_and_attend(lens, Hk, G, P, d, keep, dtype):
    case = _select_case(lens, Hk, G, P, d, dtype, 71 + d)
    cache, table, lens_, cu, q = case
    g = cache.cuda()
    sel, count = _fa().kv_page_select(q.cuda(), g[4], g[2], _i32(table), _i32(lens), P, keep)
    _ok()
    want, n = ref.select(cache, q.double().numpy(), table, lens, keep)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    np.testing.assert_array_equal(count.cpu().numpy(), n)
    for splits in (0, 1, 3, 4):
        out, lse = _fa().paged_attention_forward(q.cuda(), *g[:4], _i32(table), _i32(lens), selected=sel,
                                                 selected_count=count, num_splits=splits)
        _ok()
        _check_attend(case, out, lse, selected=[[set(w[w >= 0]) and list(w[w >= 0]) for w in r] for r in want])


def test_select_ties_go_to_the_lowest_page():
    """Equal bounds everywhere: the first pages and the last one are kept; one larger page wins."""
    P, d, n = 16, 64, 700
    case = _select_case([n * P], 1, 2, P, d, "fp16", 72)
    cache, table, lens, cu, q = case
    cache.bounds[...] = 3
    cache.scale["k"][...] = 0.25
    for special in (None, 650):
        if special is not None:
            cache.bounds[table[0, special]] = 4 * np.sign(np.where(q[0, 0].double().numpy() > 0, 1, -1))
        g = cache.cuda()
        sel, _ = _fa().kv_page_select(q.cuda(), g[4], g[2], _i32(table), _i32(lens), P, 40)
        want, _ = ref.select(cache, q.double().numpy(), table, lens, 40)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)


def test_select_special_queries_and_bad_pages():
    fa = _fa()
    case = _select_case([2000, 2000, 2000, 2000], 1, 2, 16, 64, "bf16", 73)
    cache, table, lens, cu, q = case
    q[0, 0] = 0
    q[1, 0, 3] = math.nan
    q[2, 1] *= 1e-30
    g = cache.cuda()
    sel, count = fa.kv_page_select(q.cuda(), g[4], g[2], _i32(table), _i32(lens), 16, 9)
    _ok()
    want, n = ref.select(cache, q.double().numpy(), table, lens, 9)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    table[3, 50] = cache.pages + 5
    fa.kv_page_select(q.cuda(), g[4], g[2], _i32(table), _i32(lens), 16, 9)
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
    _ok()


# ------------------------------------------------- the operators together
def test_a_server_runs_steps_in_a_graph():
    """Tables, append, attention, page choice and sparse attention of decode steps, captured once and
    replayed; every step's result against the definitions."""
    torch, fa = _torch(), _fa()
    Hk, G, P, d, B, M, keep = 2, 4, 16, 64, 5, 12, 4
    rng = np.random.default_rng(81)
    cache = ref.Cache(B * M, Hk, P, d, 81, random=False)
    g = cache.cuda()
    table, free = _i32(np.full((B, M), -1)), _i32(rng.permutation(B * M))
    h_table, h_free, h_count = table.cpu().numpy().astype(np.int64), free.cpu().numpy().astype(np.int64), B * M
    h_lens = np.zeros(B, np.int64)
    lens, count = _i32(h_lens), _i32([h_count])

    # prompts, outside of the graph
    new = np.array([37, 16, 3, 60, 1])
    T = int(new.sum())
    kv = torch.from_numpy(rng.standard_normal((2, T, Hk, d))).bfloat16()
    q = torch.from_numpy(rng.standard_normal((T, Hk * G, d))).bfloat16()
    slots, cu, lens, count, status = fa.kv_tables_step(_i32(new), lens, table, free, count, P, T, check=True)
    fa.kv_cache_append(kv[0].cuda(), kv[1].cuda(), slots, *g[:4], k_bounds=g[4])
    out, lse = fa.paged_attention_forward(q.cuda(), *g[:4], table, lens, cu_q=cu, max_q=60)
    want = ref.tables_step(new, h_lens, h_table, h_free, h_count, P, T)
    h_lens, h_table, h_free, h_count = want["lens"], want["table"], want["free"], want["count"]
    cache.append(*(x.double().numpy() for x in kv), want["slots"])
    _ok()
    _same_cache(g, cache)
    _check_attend((cache, h_table, h_lens, want["cu"], q), out, lse)

    # one decode step, captured
    s_new, s_lens, s_count = _i32(np.ones(B)), lens.clone(), count.clone()
    s_kv = torch.zeros((2, B, Hk, d), dtype=torch.bfloat16, device="cuda")
    s_q = torch.zeros((B, Hk * G, d), dtype=torch.bfloat16, device="cuda")

    def step():
        slots, cu, l, c, status = fa.kv_tables_step(s_new, s_lens, table, free, s_count, P, B)
        fa.kv_cache_append(s_kv[0], s_kv[1], slots, *g[:4], k_bounds=g[4])
        full = fa.paged_attention_forward(s_q, *g[:4], table, l, num_splits=3)
        sel, n = fa.kv_page_select(s_q, g[4], g[2], table, l, P, keep)
        part = fa.paged_attention_forward(s_q, *g[:4], table, l, selected=sel, selected_count=n)
        s_lens.copy_(l)
        s_count.copy_(c)
        return full, sel, part

    keep_state = [x.clone() for x in (*g, table, free, s_lens, s_count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # outside of the capture first; then everything as it was
        for a, b in zip((*g, table, free, s_lens, s_count), keep_state):
            a.copy_(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        full, sel, part = step()
    for _ in range(20):
        x = torch.from_numpy(rng.standard_normal((2, B, Hk, d))).bfloat16()
        y = torch.from_numpy(rng.standard_normal((B, Hk * G, d))).bfloat16()
        s_kv.copy_(x)
        s_q.copy_(y)
        graph.replay()
        _ok()
        want = ref.tables_step(np.ones(B, np.int64), h_lens, h_table, h_free, h_count, P, B)
        h_lens, h_table, h_free, h_count = want["lens"], want["table"], want["free"], want["count"]
        cache.append(*(t.double().numpy() for t in x), want["slots"])
        _same_cache(g, cache)
        case = (cache, h_table, h_lens, np.arange(B + 1), y)
        _check_attend(case, *full)
        pick, _ = ref.select(cache, y.double().numpy(), h_table, h_lens, keep)
        np.testing.assert_array_equal(sel.cpu().numpy(), pick)
        _check_attend(case, *part, selected=[[list(w[w >= 0]) for w in r] for r in pick])


def test_two_streams_at_once():
    torch, fa = _torch(), _fa()
    cases = [_attend_case([700, 300], [1, 1], 2, 4, 16, 128, "bf16", 91),
             _attend_case([500, 90, 40], [30, 1, 2], 1, 8, 32, 64, "fp16", 92)]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for case, s in zip(cases, streams):
        news = np.diff(case[3])
        g = case[0].cuda()
        args = (_i32(case[1]), _i32(case[2]))
        qd, cu = case[4].cuda(), _i32(case[3])
        torch.cuda.synchronize()
        got.append((g, args, qd, cu, fa.paged_attention_forward(qd, *g[:4], *args, cu_q=cu, max_q=int(news.max()),
                                                                 num_splits=3, stream=s)))
    torch.cuda.synchronize()
    _ok()
    for case, x in zip(cases, got):
        _check_attend(case, *x[4])


def test_the_raw_stream_handle_and_given_workspace():
    torch, fa = _torch(), _fa()
    case = _attend_case([400, 90], [1, 1], 2, 4, 16, 128, "bf16", 93)
    g = case[0].cuda()
    nbytes = 2 * 8 * 3 * 128 * 4 + 2 * 8 * 3 * 4
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    args = (case[4].cuda(), *g[:4], _i32(case[1]), _i32(case[2]))
    torch.cuda.synchronize()
    out, lse = fa.paged_attention_forward(*args, num_splits=3, workspace=ws, stream=s.cuda_stream, check=True)
    _check_attend(case, out, lse)
    with pytest.raises(fa.FaError):
        fa.paged_attention_forward(*args, num_splits=3, workspace=ws[:nbytes - 16])


def test_wrappers_refuse_wrong_tensors():
    torch, fa = _torch(), _fa()
    case = _select_case([40, 20], 2, 2, 16, 64, "bf16", 94)
    g = case[0].cuda()
    good = dict(q=case[4].cuda(), k_cache=g[0], v_cache=g[1], k_scale=g[2], v_scale=g[3], block_table=_i32(case[1]),
                lens=_i32(case[2]))
    fa.paged_attention_forward(**good)
    wrong = [dict(q=good["q"].float()), dict(q=good["q"][:1]), dict(q=good["q"].transpose(1, 2)), dict(k_cache=g[0].view(torch.uint8)),
             dict(k_cache=g[0][:, :1]), dict(v_cache=g[1][:-1]), dict(k_scale=g[2].double()), dict(v_scale=g[3][:, :1]),
             dict(block_table=good["block_table"].long()), dict(lens=good["lens"][:1]), dict(lens=good["lens"].cpu()),
             dict(out=torch.empty_like(good["q"])[:, :2]), dict(lse=torch.empty((2, 4), dtype=torch.float64, device="cuda")),
             dict(cu_q=_i32([0, 1])), dict(selected=_i32(np.zeros((2, 2, 3)))), dict(selected_count=_i32(np.zeros((2, 2)))),
             dict(scale=-1.0), dict(num_splits=65), dict(max_q=2), dict(num_splits=3, workspace=torch.empty(8, device="cuda"))]
    for w in wrong:
        with pytest.raises((TypeError, ValueError, fa.FaError)):
            fa.paged_attention_forward(**{**good, **w})
    kv = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    app = dict(k=kv, v=kv, slots=_i32([0, 1, 2]), k_cache=g[0], v_cache=g[1], k_scale=g[2], v_scale=g[3], k_bounds=g[4])
    for w in [dict(v=kv.half()), dict(v=kv[:2]), dict(k=kv[:, :1]), dict(slots=_i32([0, 1])), dict(slots=app["slots"].long()),
              dict(k_bounds=g[4][:1]), dict(k=kv[:, :, ::2])]:
        with pytest.raises((TypeError, ValueError, fa.FaError)):
            fa.kv_cache_append(**{**app, **w})
    for w in [dict(page_size=20), dict(num_selected=0), dict(q=good["q"][:1]), dict(k_bounds=g[4][:, :, :1])]:
        with pytest.raises((TypeError, ValueError, fa.FaError)):
            fa.kv_page_select(**{**dict(q=good["q"], k_bounds=g[4], k_scale=g[2], block_table=good["block_table"],
                                        lens=good["lens"], page_size=16, num_selected=2), **w})
    _ok()


def test_steps_back_to_back_equal_steps_one_by_one():
    """The kernels of a step may be set up while the one before still runs: forty steps without a wait
    give bit for bit what they give with a wait behind every call."""
    torch, fa = _torch(), _fa()
    B, Hk, G, P, d, M, steps = 96, 4, 4, 16, 128, 24, 40
    rng = np.random.default_rng(95)
    start = rng.integers(1, 300, B)
    kv = torch.from_numpy(rng.standard_normal((steps, 2, B, Hk, d)).astype(np.float32)).bfloat16().cuda()
    q = torch.from_numpy(rng.standard_normal((steps, B, Hk * G, d)).astype(np.float32)).bfloat16().cuda()
    T0 = int(start.sum())
    kv0 = torch.from_numpy(rng.standard_normal((2, T0, Hk, d)).astype(np.float32)).bfloat16().cuda()
    perm = rng.permutation(B * M)

    def run(wait):
        g = ref.Cache(B * M, Hk, P, d, random=False).cuda()
        table, free, count, lens = _i32(np.zeros((B, M))), _i32(perm), _i32([B * M]), _i32(np.zeros(B))
        one, got = _i32(np.ones(B)), []
        slots, cu, lens, count, _ = fa.kv_tables_step(_i32(start), lens, table, free, count, P, T0)
        fa.kv_cache_append(kv0[0], kv0[1], slots, *g[:4], k_bounds=g[4])
        torch.cuda.synchronize()
        for i in range(steps):
            slots, cu, lens, count, _ = fa.kv_tables_step(one, lens, table, free, count, P, B)
            wait()
            fa.kv_cache_append(kv[i, 0], kv[i, 1], slots, *g[:4], k_bounds=g[4])
            wait()
            sel, n = fa.kv_page_select(q[i], g[4], g[2], table, lens, P, 6)
            wait()
            a = fa.paged_attention_forward(q[i], *g[:4], table, lens)
            wait()
            b = fa.paged_attention_forward(q[i], *g[:4], table, lens, selected=sel, selected_count=n)
            wait()
            got += [sel, n, *a, *b]
        torch.cuda.synchronize()
        _ok()
        return got + list(g[:4]) + [g[4], table, free, lens, count]

    for x, y in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
