"""Rotary positions (include/fa_rotary.h) on the GPU: alone, turned back, and on the way into the paged 8-bit cache,
against their definitions (tests/latent_ref.py, tests/paged_ref.py).  The operators define every rounding, so most
comparisons are of bits."""
import numpy as np
import pytest

from tests import latent_ref as lref
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


_torch, _fa, _i32, _ok, _dt = base._torch, base._fa, base._i32, base._ok, base._dt


def _f32(t):
    return t.float().cpu().numpy()


def _rand(shape, dtype, seed):
    torch = _torch()
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(_dt(dtype))


def _bits(t):
    return t.view(_torch().int16)


def _want(x, pos, tab, interleaved, inverse, dtype):
    return _torch().from_numpy(lref.turn(_f32(x), pos, tab, interleaved, inverse)).to(_dt(dtype)).cuda()


@pytest.mark.parametrize("T,Hq,Hk,d,dim", [(1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (3, 5, 1, 96, 32), (7, 3, 3, 80, 80), (65, 4, 2, 256, 256),
                                            (130, 2, 1, 24, 16), (2, 1, 1, 512, 512), (9000, 40, 9, 64, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_embed(T, Hq, Hk, d, dim, dtype, interleaved):
    torch, fa = _torch(), _fa()
    rng = np.random.default_rng(T + d)
    tab = lref.table(300, dim, factor=1.25)
    pos = rng.integers(-1, 300, T)
    qkv = _rand((T, Hq + 2 * Hk, d), dtype, T * 3 + d).cuda()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    before = qkv.clone()
    for inverse in (False, True):
        qo, ko = fa.rotary_embed(q, k, _i32(pos), torch.from_numpy(tab).cuda(), interleaved=interleaved, inverse=inverse, check=True)
        for got, x in ((qo, q), (ko, k)):
            want = _want(x, pos, tab, interleaved, inverse, dtype)
            assert got.is_contiguous() and torch.equal(_bits(got), _bits(want))
            # and near the formula in 64 bits: the two products and the sum are each off by 2^-24 of their size, together
            # 2^-24 (|a cos| + |b sin| + |y|) <= 2^-24 2 sqrt(2) 1.25 max < 2^-22 1.25 max; then half a step of the type
            exact = lref.turn(_f32(x), pos, tab, interleaved, inverse, np.float64)
            f = torch.finfo(_dt(dtype))
            near = 2.0 ** -22 * np.abs(_f32(x)).max() * 1.25
            tol = near + (np.abs(exact) + near) * f.eps / 2 + f.smallest_normal * f.eps / 2
            assert (np.abs(_f32(got).astype(np.float64) - exact) <= tol).all()
    assert torch.equal(_bits(qkv), _bits(before))      # inputs stay as they were
    qo, none = fa.rotary_embed(q, None, _i32(pos), torch.from_numpy(tab).cuda(), interleaved=interleaved)
    assert none is None and torch.equal(_bits(qo), _bits(_want(q, pos, tab, interleaved, False, dtype)))
    _ok()


def test_inverse_is_the_gradient():
    """<turn(x), g> = <x, turn back(g)>, and against differences of the formula."""
    torch, fa = _torch(), _fa()
    T, H, d, dim = 11, 3, 64, 32
    tab = lref.table(40, dim, factor=1.5)
    pos = np.arange(T) * 3
    g = _rand((T, H, d), "fp16", 5)
    for inter in (False, True):
        gx, _ = fa.rotary_embed(g.cuda(), None, _i32(pos), torch.from_numpy(tab).cuda(), interleaved=inter, inverse=True, check=True)
        x = torch.randn((T, H, d), dtype=torch.float64, generator=torch.Generator().manual_seed(6)).numpy()
        e = 2.0 ** -10
        for t, h, c in ((0, 0, 0), (3, 1, 7), (10, 2, 31), (5, 0, 16), (4, 1, 50)):
            hi, lo = x.copy(), x.copy()
            hi[t, h, c] += e
            lo[t, h, c] -= e
            diff = ((lref.turn(hi, pos, tab, inter, dtype=np.float64) - lref.turn(lo, pos, tab, inter, dtype=np.float64)) / (2 * e) * g.double().numpy()).sum()
            # linear, so differences are exact but for 64-bit roundings; the operator's are two of fp32 and half a step of fp16
            got = gx[t, h, c].item()
            assert abs(got - diff) <= abs(diff) * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -20


def test_in_place_strides_and_padding():
    torch, fa = _torch(), _fa()
    T, H, d, dim = 50, 6, 96, 64
    tab, pos = lref.table(64, dim), np.arange(T) % 60 - 1
    x = _rand((T, 2, H, d + 8), "bf16", 8).cuda()
    want = x.clone()
    want[:, 1, :, :d] = _want(x[:, 1, :, :d], pos, tab, False, False, "bf16")
    v = x[:, 1, :, :d]
    a, b = fa.rotary_embed(v, None, _i32(pos), torch.from_numpy(tab).cuda(), q_out=v, check=True)
    assert a is v and torch.equal(_bits(x), _bits(want))
    # head-major memory, into a given strided output
    y = _rand((H, T, d), "bf16", 9).cuda().transpose(0, 1)
    out = torch.full((T, H + 1, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    got, k = fa.rotary_embed(y, y[:, :2], _i32(pos), torch.from_numpy(tab).cuda(), q_out=out[:, 1:, d:])
    assert torch.equal(_bits(got), _bits(_want(y, pos, tab, False, False, "bf16"))) and torch.equal(_bits(k), _bits(got[:, :2].contiguous()))
    assert (out[:, 0] == 7).all() and (out[:, :, :d] == 7).all()
    _ok()


def test_special_values_and_bad_positions():
    torch, fa = _torch(), _fa()
    x = _rand((6, 2, 32), "bf16", 10)
    x[0, 0, 0], x[1, 1, 17], x[2, 0, 31], x[3, 1, 20] = np.inf, np.nan, -np.inf, np.inf
    tab = lref.table(5, 32)
    pos = np.array([-1, 1, 2, 4, 5, -(1 << 31)])
    got, _ = fa.rotary_embed(x.cuda(), None, _i32(pos), torch.from_numpy(tab).cuda())
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG     # position 5 of 5
    want = _want(x, pos, tab, False, False, "bf16")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(3.0, 1e9, -1e9), want.nan_to_num(3.0, 1e9, -1e9))
    assert torch.equal(_bits(got[[0, 4, 5]]), _bits(x[[0, 4, 5]].cuda()))   # not turned: the same bits
    with pytest.raises(fa.FaError):
        fa.rotary_embed(x.cuda(), None, _i32(pos), torch.from_numpy(tab).cuda(), check=True)
    _ok()
    # no token at all
    a, b = fa.rotary_embed(x[:0].cuda(), x[:0].cuda(), _i32([]), torch.from_numpy(tab).cuda(), check=True)
    assert a.shape == b.shape == (0, 2, 32)


def test_rotary_wrong_tensors():
    torch, fa = _torch(), _fa()
    x, pos, tab = _rand((4, 2, 64), "bf16", 11).cuda(), _i32([0, 1, 2, 3]), torch.from_numpy(lref.table(9, 32)).cuda()
    for args in ((x, x[:3], pos, tab), (x, x[..., :32], pos, tab), (x, None, pos[:3], tab), (x, None, pos.long(), tab), (x, None, pos, tab.double()),
                 (x, None, pos, tab[0]), (x[0], None, pos, tab), (x.transpose(1, 2), None, pos, tab), (x, None, pos, tab[:, ::2])):
        with pytest.raises((ValueError, fa.FaError)):
            fa.rotary_embed(*args)
    for kw in (dict(q_out=x[:3]), dict(k_out=x), dict(q_out=x.cpu())):
        with pytest.raises(ValueError):
            fa.rotary_embed(x, None, pos, tab, **kw)
    with pytest.raises(ValueError):   # its input's memory in another order
        fa.rotary_embed(x.view(2, 4, 64)[:, :2], None, pos[:2], tab, q_out=x[:2])
    for y in (x.float(), x.to(torch.float8_e4m3fn)):
        with pytest.raises(TypeError):
            fa.rotary_embed(y, None, pos, tab)
    with pytest.raises(TypeError):
        fa.rotary_embed(x, x.half(), pos, tab)
    with pytest.raises(fa.FaError):   # more channels than a head has
        fa.rotary_embed(x[..., :16], None, pos, tab)
    with pytest.raises(fa.FaError):   # one head for all: not a stride
        fa.rotary_embed(x[:, :1].expand(4, 3, 64), None, pos, tab)
    _ok()


# --------------------------------------------------------- into the cache
def _append_case(Hk, G, P, d, dim, dtype, news, lens, seed, inter, bounds=True, pad=3):
    """A cache with tokens, then new ones that begin inside pages; returns what is needed to call and to compare."""
    torch = _torch()
    rng = np.random.default_rng(seed)
    have = -(-(np.array(lens) + news) // P)
    pages = int(have.sum()) + 2
    cache = ref.Cache(pages, Hk, P, d, seed=seed)
    perm = rng.permutation(pages)
    slots, pos, at = [], [], 0
    for b, (n, l) in enumerate(zip(news, lens)):
        row = perm[at:at + have[b]]
        at += have[b]
        j = np.arange(l, l + n)
        slots.append(row[j // P] * P + j % P)
        pos.append(j)
        for i, page in enumerate(row):
            cache.set_bounds(page, max(1, min(P, l - i * P)))
    slots, pos = np.concatenate(slots + [np.full(pad, -1)]), np.concatenate(pos + [np.full(pad, -1)])
    T = len(slots)
    qkv = (torch.randn((T, Hk * G + 2 * Hk, d), generator=torch.Generator().manual_seed(seed)) *
           torch.exp(torch.randn((T, Hk * G + 2 * Hk, 1), generator=torch.Generator().manual_seed(seed + 1)))).to(_dt(dtype)).cuda()
    tab = lref.table(max(int(pos.max()) + 1, 1), dim, factor=1.1)
    return cache, qkv, slots, pos, tab


def _check_cache(g, cache, bounds):
    codes = [x.view(_torch().uint8).cpu().numpy() for x in g[:2]]
    for c, n in zip(codes, "kv"):
        want = cache.codes[n]
        nan = np.isnan(ref.VALUES[want])
        assert np.array_equal(c[~nan], want[~nan]) and np.isnan(ref.VALUES[c[nan]]).all()
    for s, n in zip(g[2:4], "kv"):
        np.testing.assert_array_equal(s.double().cpu().numpy(), cache.scale[n])
    if bounds:
        np.testing.assert_array_equal(g[4].cpu().numpy(), cache.bounds)


@pytest.mark.parametrize("Hk,G,P,d,dim,news,lens", [
    (1, 1, 16, 16, 16, [1], [0]), (2, 4, 64, 128, 128, [1, 1, 1], [5, 64, 200]), (8, 4, 64, 128, 64, [70, 1, 130], [3, 63, 0]),
    (3, 2, 32, 80, 80, [9, 40], [30, 0]), (2, 1, 128, 256, 256, [300, 2], [100, 127]), (5, 1, 128, 96, 32, [128, 1], [0, 9]),
    (1, 2, 16, 64, 48, [5, 5, 33, 1], [11, 12, 15, 16])])
@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("fp16", True), ("bf16", True)])
def test_append_rotary(Hk, G, P, d, dim, news, lens, dtype, inter):
    """Codes, scales, bounds and queries, bit for bit."""
    torch, fa = _torch(), _fa()
    for bounds in (True, False):
        cache, qkv, slots, pos, tab = _append_case(Hk, G, P, d, dim, dtype, news, lens, 31 + d + P, inter)
        q, k, v = qkv[:, :Hk * G], qkv[:, Hk * G:Hk * G + Hk], qkv[:, Hk * G + Hk:]
        g = cache.cuda()
        got = fa.kv_cache_append_rotary(q, k, v, _i32(pos), torch.from_numpy(tab).cuda(), _i32(slots), *g[:4],
                                        k_bounds=g[4] if bounds else None, interleaved=inter, check=True)
        cache.append(lref.turn(_f32(k), pos, tab, inter).astype(np.float64), _f32(v).astype(np.float64), slots, bounds)
        _check_cache(g, cache, bounds)
        assert torch.equal(_bits(got), _bits(_want(q, pos, tab, inter, False, dtype)))
    # without queries, and with them in place
    cache, qkv, slots, pos, tab = _append_case(Hk, G, P, d, dim, dtype, news, lens, 31 + d + P, inter)
    g2 = cache.cuda()
    assert fa.kv_cache_append_rotary(None, k, v, _i32(pos), torch.from_numpy(tab).cuda(), _i32(slots), *g2[:4], interleaved=inter) is None
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(g[:2], g2[:2]))
    qq = q.clone()
    assert fa.kv_cache_append_rotary(qq, k, v, _i32(pos), torch.from_numpy(tab).cuda(), _i32(slots), *cache.cuda()[:4], interleaved=inter, q_out=qq) is qq
    assert torch.equal(_bits(qq), _bits(got))
    _ok()


def test_append_rotary_odd_rows():
    """Rows left out between a page's tokens, tokens without a position, positions beyond the table (reported, stored
    as they are), special values."""
    torch, fa = _torch(), _fa()
    Hk, P, d, dim = 2, 16, 64, 32
    cache = ref.Cache(4, Hk, P, d, seed=3)
    slots = np.array([0, -1, 1, 2, -1, -1, 3, 32, 33, 34])
    pos = np.array([0, 5, 1, -1, 7, 9, 3, 100, 2, 4])
    tab = lref.table(10, dim)
    kv = _rand((10, 2, Hk, d), "bf16", 12)
    kv[0, 0, 0, 3], kv[2, 0, 1, 5], kv[8, 1, 0, 1] = np.nan, np.inf, -np.inf
    g = cache.cuda()
    fa.kv_cache_append_rotary(None, kv[:, 0].cuda(), kv[:, 1].cuda(), _i32(pos), torch.from_numpy(tab).cuda(), _i32(slots), *g[:4], k_bounds=g[4])
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
    # the oracle takes a page's tokens one after the other: without the rows that are left out
    on = slots >= 0
    k = lref.turn(_f32(kv[:, 0]), np.where(pos < 10, pos, -1), tab, False).astype(np.float64)
    cache.append(k[on], _f32(kv[:, 1]).astype(np.float64)[on], slots[on], True)
    _check_cache(g, cache, True)
    _ok()


def test_append_rotary_refusals():
    torch, fa = _torch(), _fa()
    g = ref.Cache(4, 2, 16, 64, seed=1).cuda()
    x, i, tab = _rand((3, 2, 64), "bf16", 13).cuda(), _i32([0, 1, 2]), torch.from_numpy(lref.table(9, 32)).cuda()
    for args in ((x[:2], x, x, i, tab, i), (x[..., :32], x, x, i, tab, i), (x, x[:, :1], x, i, tab, i), (x, x, x[:2], i, tab, i), (x, x, x, i[:2], tab, i),
                 (x, x, x, i, tab, i[:2]), (x, x, x, i, tab.half(), i)):
        with pytest.raises(ValueError):
            fa.kv_cache_append_rotary(*args, *g[:4])
    with pytest.raises(ValueError):
        fa.kv_cache_append_rotary(None, x, x, i, tab, i, *g[:4], q_out=x)
    with pytest.raises(TypeError):
        fa.kv_cache_append_rotary(x.half(), x, x, i, tab, i, *g[:4])
    with pytest.raises(fa.FaError):
        fa.kv_cache_append_rotary(x, x, x, i, torch.from_numpy(lref.table(9, 80)).cuda(), i, *g[:4])
    none = x[:0]
    assert fa.kv_cache_append_rotary(none, none, none, i[:0], tab, i[:0], *g[:4], check=True).shape == (0, 2, 64)


def test_step_turned_and_stored_then_read():
    """Tables, the turning append and attention over the cache, two steps of them captured in a graph and replayed, on
    another stream than the current one."""
    torch, fa = _torch(), _fa()
    Hk, G, P, d, dim, B = 2, 4, 32, 64, 64, 3
    lens0, news = np.array([0, 40, 31]), [np.array([37, 1, 5]), np.array([1, 1, 1])]
    pages = 12
    cache = ref.Cache(pages, Hk, P, d, random=False)
    table, free, at = np.zeros((B, 4), np.int64), np.arange(pages), pages
    for b in range(B):
        for j in range(-(-lens0[b] // P)):
            at -= 1
            table[b, j] = free[at]
    full = ref.Cache(pages, Hk, P, d, seed=21)
    for n in "kv":
        cache.codes[n], cache.scale[n] = full.codes[n], full.scale[n]
    tab = lref.table(100, dim)
    T = [int(n.sum()) + 2 for n in news]
    qkv = [_rand((t, Hk * G + 2 * Hk, d), "bf16", 14 + i).cuda() for i, t in enumerate(T)]
    s = torch.cuda.Stream()
    g, gt, gf, gl, gc = cache.cuda(), _i32(table), _i32(free), _i32(lens0), _i32([at])
    start = [x.clone() for x in (*g[:4], gt, gf)]
    dev_tab, new_t = torch.from_numpy(tab).cuda(), [_i32(n) for n in news]

    def step(i, lens, count):
        slots, cu, lens, count, _ = fa.kv_tables_step(new_t[i], lens, gt, gf, count, P, T[i])
        row = torch.searchsorted(cu, torch.arange(T[i], device="cuda", dtype=torch.int32), right=True, out_int32=True) - 1
        row = row.clamp(max=B - 1)
        pos = torch.where(slots >= 0, lens[row.long()] - (cu[row.long() + 1] - torch.arange(T[i], device="cuda")), -1).int()
        x = qkv[i]
        q = fa.kv_cache_append_rotary(x[:, :Hk * G], x[:, Hk * G:Hk * G + Hk], x[:, Hk * G + Hk:], pos, dev_tab, slots, *g[:4])
        out, lse = fa.paged_attention_forward(q, *g[:4], gt, lens, cu_q=cu, max_q=int(news[i].max()))
        return lens, count, out, lse, slots, pos

    with torch.cuda.stream(s):
        l, c, *_ = step(0, gl, gc)
        step(1, l, c)
        for x, y in zip((*g[:4], gt, gf), start):
            (x.view(torch.uint8) if x.dtype == ref.E4M3 else x).copy_(y.view(torch.uint8) if y.dtype == ref.E4M3 else y)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            l, c, *one = step(0, gl, gc)
            l, c, *two = step(1, l, c)
        graph.replay()
        s.synchronize()
    _ok()
    tb, fr, count, lens = table, free, at, lens0
    for i, got in enumerate((one, two)):
        r = ref.tables_step(news[i], lens, tb, fr, count, P, T[i])
        tb, fr, count, lens = r["table"], r["free"], r["count"], r["lens"]
        np.testing.assert_array_equal(got[2].cpu().numpy(), r["slots"])
        pos = got[3].cpu().numpy()
        x = _f32(qkv[i])
        k = lref.turn(x[:, Hk * G:Hk * G + Hk], pos, tab, False).astype(np.float64)
        cache.append(k, x[:, Hk * G + Hk:].astype(np.float64), r["slots"], False)
        q = _want(qkv[i][:, :Hk * G], pos, tab, False, False, "bf16").double().cpu().numpy()
        want = ref.attend(cache, q, tb, lens, r["cu"], d ** -0.5, True)
        v_top = max(np.abs(cache.request(tb[b], int(lens[b]), "v")).max() for b in range(B))
        ref.check(got[0], got[1], want, d, int(lens.max()), v_top, torch.bfloat16, rows=slice(0, int(r["cu"][-1])))


@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("fp16", True)])
def test_append_rotary_many_queries(dtype, inter):
    """Queries enough (1024 items per SM) for a launch of their own: into new memory, and in place beside the keys and values."""
    torch, fa = _torch(), _fa()
    Hk, G, P, d, dim = 8, 4, 64, 64, 48
    for in_place in (False, True):
        cache, qkv, slots, pos, tab = _append_case(Hk, G, P, d, dim, dtype, [900, 400], [5, 0], 51, inter)
        before = qkv.clone()
        q, k, v = qkv[:, :Hk * G], qkv[:, Hk * G:Hk * G + Hk], qkv[:, Hk * G + Hk:]
        want = _want(q, pos, tab, inter, False, dtype)
        g = cache.cuda()
        got = fa.kv_cache_append_rotary(q, k, v, _i32(pos), torch.from_numpy(tab).cuda(), _i32(slots), *g[:4], k_bounds=g[4],
                                        interleaved=inter, q_out=q if in_place else None, check=True)
        cache.append(lref.turn(_f32(k), pos, tab, inter).astype(np.float64), _f32(v).astype(np.float64), slots, True)
        _check_cache(g, cache, True)
        assert torch.equal(_bits(got), _bits(want)) and (got is q) == in_place
        assert torch.equal(_bits(qkv[:, Hk * G:]), _bits(before[:, Hk * G:]))
        assert in_place or torch.equal(_bits(qkv), _bits(before))
    _ok()


def test_in_place_through_a_view_with_other_unused_strides():
    """One token's queries within a joint projection and a view of the same memory: the token stride is never used."""
    torch, fa = _torch(), _fa()
    tab, pos = lref.table(9, 32), np.array([7])
    qkv = _rand((1, 12, 32), "bf16", 52).cuda()
    q, want = qkv[:, :4], qkv.clone()
    want[:, :4] = _want(q, pos, tab, False, False, "bf16")
    view = q.as_strided((1, 4, 32), (4 * 32, 32, 1))
    assert view.stride() != q.stride() and view.data_ptr() == q.data_ptr()
    got, _ = fa.rotary_embed(q, None, _i32(pos), torch.from_numpy(tab).cuda(), q_out=view, check=True)
    assert got is view and torch.equal(_bits(qkv), _bits(want))
