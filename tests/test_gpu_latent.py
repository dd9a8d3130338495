"""Latent attention (include/fa_latent.h) on the GPU against its definition in 64 bits (tests/latent_ref.py)."""
import math

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


def _rand(shape, dtype, seed, size=1.0):
    torch = _torch()
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * size).to(_dt(dtype))


def _f64(t):
    return t.double().cpu().numpy()


def _bits(t):
    return t.contiguous().view(_torch().int16)


# ------------------------------------------------------------ the cache's rows
@pytest.mark.parametrize("C,R,H,T,P", [(512, 64, 128, 3, 64), (512, 64, 16, 700, 16), (8, 16, 1, 1, 128), (256, 32, 5, 37, 32), (72, 48, 3, 300, 16)])
@pytest.mark.parametrize("dtype,inter", [("bf16", True), ("fp16", False)])
def test_latent_append(C, R, H, T, P, dtype, inter):
    """Rows bit for bit, turned and as they are; other rows of the cache stay."""
    torch, fa = _torch(), _fa()
    rng = np.random.default_rng(C + T)
    pages = -(-T // P) + 3
    slots = rng.permutation(pages * P)[:T]
    slots[rng.random(T) < 0.1] = -1
    pos = np.where(rng.random(T) < 0.1, -1, rng.integers(0, 90, T))
    tab = lref.table(90, R)
    kv, q = _rand((T, C + R + 8), dtype, 1).cuda(), _rand((T, H, R + 24), dtype, 2).cuda()
    latent, rope, qr = kv[:, :C], kv[:, C:C + R], q[..., 24:]
    cache = _rand((pages, P, C + R), dtype, 3).cuda()
    for turned in (True, False):
        got = cache.clone()
        kw = dict(q_rope=qr, positions=_i32(pos), table=torch.from_numpy(tab).cuda(), interleaved=inter) if turned else {}
        out = fa.latent_cache_append(latent, rope, _i32(slots), got, check=True, **kw)
        want, on = cache.view(-1, C + R).clone(), slots >= 0
        k = torch.from_numpy(lref.turn(rope.float().cpu().numpy()[:, None], pos, tab, inter)[:, 0]).to(_dt(dtype)).cuda() if turned else rope
        want[slots[on]] = torch.cat([latent, k], dim=1)[torch.from_numpy(on).cuda()]
        assert torch.equal(_bits(got.view(-1, C + R)), _bits(want))
        if turned:
            wq = torch.from_numpy(lref.turn(qr.float().cpu().numpy(), pos, tab, inter)).to(_dt(dtype)).cuda()
            assert torch.equal(_bits(out), _bits(wq))
            wide = torch.full((T, H, C + R), 5.0, dtype=_dt(dtype), device="cuda")
            assert fa.latent_cache_append(latent, rope, _i32(slots), got, q_out=wide[..., C:], **kw).data_ptr() == wide[..., C:].data_ptr()
            assert torch.equal(_bits(wide[..., C:]), _bits(wq)) and (wide[..., :C] == 5).all()
        else:
            assert out is None
    _ok()


def test_latent_append_edges():
    torch, fa = _torch(), _fa()
    cache = _rand((2, 16, 24), "bf16", 4).cuda()
    x, r = _rand((5, 8), "bf16", 5).cuda(), _rand((5, 16), "bf16", 6).cuda()
    before = cache.clone()
    fa.latent_cache_append(x, r, _i32([32, -5, 3, 1 << 30, -1]), cache)            # slots beyond the cache
    assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
    before.view(-1, 24)[3] = torch.cat([x[2], r[2]])
    assert torch.equal(_bits(cache), _bits(before))
    fa.latent_cache_append(x, r, _i32([-1] * 5), cache, check=True)
    fa.latent_cache_append(x[:0], r[:0], _i32([]), cache, check=True)
    assert torch.equal(_bits(cache), _bits(before))
    plain = _rand((2, 16, 8), "bf16", 7).cuda()
    fa.latent_cache_append(x, None, _i32([0, 1, 2, 3, 4]), plain, check=True)      # R = 0
    assert torch.equal(_bits(plain[0, :5]), _bits(x))
    i, tab = _i32([0, 1, 2, 3, 4]), torch.from_numpy(lref.table(9, 16)).cuda()
    for args, kw in (((x, r[:4], i, cache), {}), ((x, None, i, cache), {}), ((x, r, i[:4], cache), {}), ((x, r, i, cache[0]), {}), ((x, r, i, plain), {}),
                     ((x, r, i, cache), dict(q_rope=r[:, None])), ((x, r, i, cache), dict(q_out=r[:, None])),
                     ((x, r, i, cache), dict(q_rope=r[:4, None], positions=i, table=tab)), ((x.t(), r, i, cache), {})):
        with pytest.raises(ValueError):
            fa.latent_cache_append(*args, **kw)
    with pytest.raises(TypeError):
        fa.latent_cache_append(x, r.half(), i, cache)
    with pytest.raises(TypeError):
        fa.latent_cache_append(x, r, i, cache, positions=i)
    with pytest.raises(fa.FaError):
        fa.latent_cache_append(x, r, i, cache, positions=i, table=torch.from_numpy(lref.table(9, 32)).cuda())
    _ok()


# ------------------------------------------------------------ absorbed form
class Case:
    """Requests over a paged cache: places behind a request's last token, and pages of no request, hold NaN."""

    def __init__(self, lens, news, H, C, R, P, dtype, seed, size=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.news, self.H, self.C, self.W, self.P, self.dtype = np.array(lens), np.array(news), H, C, C + R, P, dtype
        have = -(-self.lens // P)
        pages = int(have.sum()) + spare
        self.cache = _rand((pages, P, C + R), dtype, seed, size)
        self.table = np.full((len(lens), max(int(have.max()), 1) + 1), 1 << 30)
        perm, at = rng.permutation(pages), 0
        self.keys = []
        used = np.zeros(pages, bool)
        for b, n in enumerate(have):
            self.table[b, :n] = perm[at:at + n]
            used[perm[at:at + n]] = True
            at += n
            if n and self.lens[b] % P:
                self.cache[perm[at - 1], self.lens[b] % P:] = math.nan
            self.keys.append(_f64(self.cache[perm[at - n:at]].reshape(-1, C + R)[:self.lens[b]]))
        self.cache[~used] = math.nan
        self.cu = np.concatenate([[0], np.cumsum(news)])
        self.q = _rand((int(self.cu[-1]), H, C + R), dtype, seed + 1)
        self.scale = 1.0 / math.sqrt(C + R)

    def call(self, **kw):
        fa = _fa()
        kw = {**dict(cu_q=_i32(self.cu), max_q=max(int(self.news.max()), 1), scale=self.scale), **kw}
        return fa.latent_paged_attention_forward(self.q.cuda(), self.cache.cuda(), _i32(self.table), _i32(self.lens), self.C, **kw)

    def want(self, causal=True):
        parts = []
        for b, (n, m) in enumerate(zip(self.news, self.lens)):
            limits = [m - n + i + 1 if causal else m for i in range(n)]
            k = self.keys[b]
            parts.append(lref.attend(_f64(self.q[self.cu[b]:self.cu[b + 1]]), k, k[:, :self.C], limits, self.scale))
        return [np.concatenate(x) for x in zip(*parts)]

    def check(self, out, lse, causal=True, rows=slice(None)):
        top = max([np.abs(k).max() for k in self.keys if k.size] + [0.0])
        lref.check(out, lse, self.want(causal), self.W, max(int(self.lens.max()), 1), top, _dt(self.dtype), rows)


@pytest.mark.parametrize("H,C,R,P,lens,news", [
    (16, 512, 64, 64, [1, 64, 63, 65, 300, 128], [1] * 6),
    (128, 512, 64, 64, [700, 1, 129, 64], [1] * 4),
    (64, 512, 64, 16, [50, 17, 16, 500], [1] * 4),
    (1, 8, 0, 128, [1, 5, 200], [1] * 3), (5, 64, 8, 32, [33, 31, 400, 1], [1] * 4), (3, 72, 16, 16, [90, 40], [1] * 2),
    (20, 256, 32, 16, [300, 77, 12], [5, 3, 1]), (65, 128, 32, 64, [200, 3], [2, 3]), (128, 512, 64, 128, [260, 90], [4, 2]),
    (7, 192, 0, 32, [150, 64], [40, 33]), (40, 320, 16, 64, [70, 200], [7, 9]), (96, 512, 64, 32, [130], [130]), (2, 448, 128, 16, [5, 80], [1, 1]),
    (33, 200, 24, 64, [129, 65], [1, 1])])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_absorbed(H, C, R, P, lens, news, dtype):
    c = Case(lens, news, H, C, R, P, dtype, 50 + H + C)
    for causal in (True, False):
        out, lse = c.call(causal=causal, check=True)
        c.check(out, lse, causal)


def test_absorbed_one_query_per_request_without_marks():
    c = Case([100, 3, 70], [1, 1, 1], 16, 128, 32, 16, "bf16", 61)
    out, lse = c.call(cu_q=None, max_q=1, check=True)
    c.check(out, lse)


@pytest.mark.parametrize("members", [(16, 1), (100, 1), (30, 7)])
def test_absorbed_requests_that_see_nothing(members):
    """No key, no query, more queries than keys: rows of zeros with LSE -inf, others as ever."""
    H, most = members
    lens, news = [0, 130, 5, 0, 64, 0], [most, most, 9, 0, 0, 1]
    c = Case(lens, news, H, 256, 64, 64, "bf16", 62)
    out, lse = c.call(check=True)
    c.check(out, lse)
    out, lse = c.call(causal=False, check=True)
    c.check(out, lse, False)
    c = Case([0, 0], [1, 1], H, 256, 64, 64, "bf16", 63)
    out, lse = c.call(check=True)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_absorbed_many_unequal_requests():
    """More units than CTAs, and shares that end anywhere."""
    rng = np.random.default_rng(64)
    lens = rng.integers(0, 400, 500)
    lens[7] = 9000
    c = Case(lens, np.ones(500, int), 8, 64, 16, 16, "bf16", 65)
    out, lse = c.call(check=True)
    c.check(out, lse)
    again = c.call()
    assert _torch().equal(_bits(again[0]), _bits(out)) and _torch().equal(again[1], lse)


def test_absorbed_long_request():
    for H, n in ((16, 1), (128, 2)):
        c = Case([70001], [n], H, 512, 64, 64, "bf16", 66)
        out, lse = c.call(check=True)
        c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("grow", [1.02, 0.98, 1.0])
def test_absorbed_moving_references(dtype, grow):
    """Scores that grow (references move again and again), fall, or are all the same."""
    torch = _torch()
    c = Case([900, 333], [2, 1], 33, 128, 64, 64, dtype, 67)
    f = torch.tensor([grow ** j for j in range(960)], dtype=torch.float64)
    base_row = _f64(c.q[0, 0])[None] * 0.25
    for b, m in enumerate(c.lens):
        k = torch.from_numpy(base_row) * f[:m, None] * (0 if grow == 1.0 else 1)
        k = k.clamp(-40, 40).to(_dt(dtype))
        pages = c.table[b, :-(-m // c.P)]
        whole = c.cache[pages].reshape(-1, c.W)
        whole[:m] = k
        c.cache[pages] = whole.reshape(-1, c.P, c.W)
        c.keys[b] = _f64(k)
    c.scale = 0.15
    out, lse = c.call(check=True)
    c.check(out, lse)


def test_absorbed_special_values():
    """A NaN or infinity in a query stays in its row; NaN behind the last key reaches nothing (every Case has that)."""
    torch = _torch()
    c = Case([100, 90], [2, 1], 20, 128, 64, 16, "bf16", 68)
    clean, _ = c.call(check=True)
    c.q[0, 3, 5], c.q[2, 19, 150], c.q[1, 0, 0] = math.nan, math.nan, math.inf
    out, lse = c.call(check=True)
    hit = torch.zeros(3, 20, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[2, 19] = hit[1, 0] = True
    assert out[hit].isnan().all() and lse[0, 3].isnan() and lse[2, 19].isnan()
    assert torch.equal(_bits(out[~hit]), _bits(clean[~hit]))


def test_absorbed_strides_given_outputs_and_rows_of_none():
    torch, fa = _torch(), _fa()
    c = Case([100, 90, 40], [3, 1, 2], 20, 128, 64, 16, "fp16", 69)
    T, H = c.q.shape[:2]
    wide = torch.full((H, T + 9, c.W + 16), 9.0, dtype=torch.float16, device="cuda")
    q = wide[:, 4:4 + T, 8:8 + c.W].transpose(0, 1)
    q.copy_(c.q)
    padded = torch.full((T + 9, H, c.W), math.nan, dtype=torch.float16, device="cuda")
    padded[4:4 + T] = q
    out = torch.full((T + 9, H, c.C + 40), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T + 9, H), 7.0, device="cuda")
    o, l = fa.latent_paged_attention_forward(padded, c.cache.cuda(), _i32(c.table), _i32(c.lens), c.C, _i32(c.cu + 4), 3, scale=c.scale,
                                             out=out[..., 16:16 + c.C], lse=lse, check=True)
    assert l is lse and o.data_ptr() == out[..., 16:].data_ptr()
    c.check(o[4:4 + T], l[4:4 + T])
    assert (out[:4] == 7).all() and (out[4 + T:] == 7).all() and (out[..., :16] == 7).all() and (out[..., 16 + c.C:] == 7).all()
    assert (lse[:4] == 7).all() and (lse[4 + T:] == 7).all()
    o, l = fa.latent_paged_attention_forward(q, c.cache.cuda(), _i32(c.table), _i32(c.lens), c.C, _i32(c.cu), 3, scale=c.scale, check=True)
    c.check(o, l)


def test_absorbed_bad_data_is_reported():
    """Bad pages, lengths and marks: reported, nothing read outside, the other requests have their outputs."""
    torch, fa = _torch(), _fa()
    for what in ("page", "negative page", "length", "negative length", "marks"):
        c = Case([200, 90, 300], [1, 2, 1], 20, 128, 64, 64, "bf16", 70)
        table, lens, cu = c.table.copy(), c.lens.copy(), c.cu.copy()
        if "page" in what:
            table[1, 0] = -3 if "negative" in what else c.cache.shape[0]
        elif "length" in what:
            lens[1] = -1 if "negative" in what else c.table.shape[1] * c.P + 1
        else:
            cu[2], lens[2] = 100, 300
        out, lse = torch.full((4, 20, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 20), 7.0, device="cuda")
        fa.latent_paged_attention_forward(c.q.cuda(), c.cache.cuda(), _i32(table), _i32(lens), c.C, _i32(cu), 2, scale=c.scale, out=out, lse=lse)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
        _ok()
        c.check(out, lse, rows=slice(0, 1))
        if what != "marks":
            c.check(out, lse, rows=slice(3, 4))


def test_absorbed_offsets_beyond_32_bits():
    """Rows behind 2^31 elements of the cache."""
    torch, fa = _torch(), _fa()
    P, C, R = 64, 512, 64
    pages = (1 << 31) // (P * (C + R)) + 40
    big = torch.empty((pages, P, C + R), dtype=torch.bfloat16, device="cuda")
    big[:3] = math.nan
    c = Case([150], [1], 16, C, R, P, "bf16", 71)
    table = np.array([[pages - 1, pages - 30, pages - 2, 0]])
    big[table[0, :3]] = c.cache[c.table[0, :3]].cuda()
    out, lse = fa.latent_paged_attention_forward(c.q.cuda(), big, _i32(table), _i32(c.lens), C, scale=c.scale, check=True)
    c.check(out, lse)
    # and written there
    x, r = _rand((1, C), "bf16", 72).cuda(), _rand((1, R), "bf16", 73).cuda()
    fa.latent_cache_append(x, r, _i32([(pages - 1) * P + 63]), big, check=True)
    assert torch.equal(_bits(big[-1, 63]), _bits(torch.cat([x[0], r[0]])))


def test_absorbed_without_a_query():
    torch, fa = _torch(), _fa()
    c = Case([10, 20], [1, 1], 4, 64, 16, 16, "bf16", 74)
    g, dev = c.cache.cuda(), (_i32(c.table), _i32(c.lens))
    none = c.q[:0].cuda()
    for max_q in (0, 1, 100):
        out, lse = fa.latent_paged_attention_forward(none, g, *dev, 64, _i32([0, 0, 0]), max_q, scale=0.1, check=True)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = fa.latent_paged_attention_forward(none, g, dev[0][:0], dev[1][:0], 64, scale=0.1, stream=torch.cuda.Stream())
    assert out.shape == (0, 4, 64)
    with pytest.raises(fa.FaError):
        fa.latent_paged_attention_forward(none, g, *dev, 64, scale=0.1)


def test_absorbed_refusals():
    torch, fa = _torch(), _fa()
    c = Case([10, 20], [1, 1], 4, 64, 16, 16, "bf16", 75)
    q, g, t, l = c.q.cuda(), c.cache.cuda(), _i32(c.table), _i32(c.lens)
    for args in ((q[..., :72], g, t, l, 64), (q, g[0], t, l, 64), (q, g, t[0], l, 64), (q, g, t, l[:1], 64), (q, g, t, l, 88), (q, g, t.long(), l, 64),
                 (q, g.half(), t, l, 64), (q, g, t, l, -8)):
        with pytest.raises(ValueError):
            fa.latent_paged_attention_forward(*args, scale=0.1)
    for kw in (dict(out=q), dict(lse=q), dict(cu_q=_i32([0, 1]))):
        with pytest.raises(ValueError):
            fa.latent_paged_attention_forward(q, g, t, l, 64, scale=0.1, **kw)
    for kw in (dict(max_q=2), dict(scale=0.0), dict(scale=math.nan)):
        with pytest.raises(fa.FaError):
            fa.latent_paged_attention_forward(q, g, t, l, 64, **{"scale": 0.1, **kw})
    with pytest.raises(TypeError):
        fa.latent_paged_attention_forward(q, g, t, l, 64)           # no scale
    with pytest.raises(fa.FaError):
        fa.latent_paged_attention_forward(q, g, t, l, 60, scale=0.1)
    long = Case([1000], [1], 4, 64, 16, 16, "bf16", 76)
    with pytest.raises(fa.FaError):                                  # a workspace that is too small
        long.call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    _ok()


# ------------------------------------------------------------ expanded form
class Ragged:
    def __init__(self, news, keys, H, Dn, R, Dv, dtype, seed):
        self.news, self.lens, self.H, self.Dn, self.R, self.Dv, self.dtype = np.array(news), np.array(keys), H, Dn, R, Dv, dtype
        self.cu_q, self.cu_k = np.concatenate([[0], np.cumsum(news)]), np.concatenate([[0], np.cumsum(keys)])
        self.q, self.kv = _rand((self.cu_q[-1], H, Dn + R), dtype, seed), _rand((self.cu_k[-1], H, Dn + Dv), dtype, seed + 1)
        self.shared = _rand((self.cu_k[-1], R), dtype, seed + 2)
        self.scale = 1.0 / math.sqrt(Dn + R)

    def args(self):
        kv = self.kv.cuda()
        return self.q.cuda(), kv[..., :self.Dn], self.shared.cuda(), kv[..., self.Dn:], _i32(self.cu_q), _i32(self.cu_k)

    def call(self, **kw):
        return _fa().latent_attention_forward(*self.args(), **{**dict(max_q=max(int(self.news.max()), 1), max_k=max(int(self.lens.max()), 1)), **kw})

    def want(self, causal=True, only=None):
        parts = []
        for b, (n, m) in enumerate(zip(self.news, self.lens)):
            rows, keys = slice(self.cu_q[b], self.cu_q[b + 1]), slice(self.cu_k[b], self.cu_k[b + 1])
            sh = np.broadcast_to(_f64(self.shared[keys])[:, None], (m, self.H, self.R))
            k = np.concatenate([_f64(self.kv[keys][..., :self.Dn]), sh], axis=2)
            parts.append(lref.attend(_f64(self.q[rows]), k, _f64(self.kv[keys][..., self.Dn:]), [m - n + i + 1 if causal else m for i in range(n)], self.scale))
        return [np.concatenate(x) for x in zip(*parts)]

    def check(self, out, lse, causal=True, rows=slice(None)):
        top = np.abs(np.nan_to_num(_f64(self.kv[..., self.Dn:]))).max(initial=0.0)
        lref.check(out, lse, self.want(causal), self.Dn + self.R, max(int(self.lens.max()), 1), top, _dt(self.dtype), rows)


@pytest.mark.parametrize("H,Dn,R,Dv,news,keys", [
    (2, 128, 64, 128, [1, 128, 129], [1, 128, 129]), (1, 128, 64, 128, [300, 17], [300, 500]), (3, 64, 32, 64, [256, 1, 200], [256, 700, 330]),
    (2, 96, 32, 80, [33, 257, 5], [40, 257, 128]), (1, 8, 8, 8, [3, 150], [9, 150]), (2, 48, 16, 112, [140, 2], [150, 130]),
    (1, 128, 64, 64, [127, 255], [640, 256]), (2, 56, 64, 24, [100], [383]), (1, 120, 8, 128, [513], [513])])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_expanded(H, Dn, R, Dv, news, keys, dtype):
    c = Ragged(news, keys, H, Dn, R, Dv, dtype, 80 + H + Dn)
    for causal in (True, False):
        out, lse = c.call(causal=causal, check=True)
        c.check(out, lse, causal)


def test_expanded_requests_that_see_nothing():
    c = Ragged([5, 0, 130, 300, 0, 7], [0, 50, 3, 20, 0, 7], 2, 128, 64, 128, "bf16", 90)
    for causal in (True, False):
        out, lse = c.call(causal=causal, check=True)
        c.check(out, lse, causal)
    c = Ragged([5, 1], [0, 0], 2, 128, 64, 128, "bf16", 91)     # no key anywhere
    out, lse = c.call(check=True)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_expanded_keys_stay_in_their_request():
    """NaN and infinities in the keys and values of one request do not reach its neighbours in the same tiles."""
    torch = _torch()
    c = Ragged([100, 60, 200, 1], [100, 70, 333, 90], 2, 128, 64, 128, "bf16", 92)
    clean, _ = c.call(check=True)
    c.check(*c.call())
    a, b = c.cu_k[1], c.cu_k[2]
    c.kv[a:b], c.shared[a:b] = math.nan, math.inf
    out, lse = c.call(check=True)
    keep = np.r_[0:c.cu_q[1], c.cu_q[2]:c.cu_q[4]]
    assert torch.equal(_bits(out[keep]), _bits(clean[keep])) and out[c.cu_q[1]:c.cu_q[2]].isnan().all()
    # and a query's NaN stays in its row
    c = Ragged([100, 60], [100, 70], 2, 64, 32, 64, "fp16", 93)
    clean, _ = c.call()
    c.q[130, 1, 70] = math.nan
    out, _ = c.call(check=True)
    assert out[130, 1].isnan().all()
    out[130, 1] = clean[130, 1]
    assert torch.equal(_bits(out), _bits(clean))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("grow", [1.01, 0.99, 1.0])
def test_expanded_moving_references(dtype, grow):
    torch = _torch()
    c = Ragged([260], [900], 2, 64, 32, 64, dtype, 94)
    f = torch.tensor([grow ** j for j in range(900)], dtype=torch.float64)[:, None, None]
    c.kv[..., :64] = ((c.q[0, :, :64].double() * 0.25)[None] * f * (grow != 1.0)).clamp(-40, 40).to(_dt(dtype))
    c.shared[:] = 0
    out, lse = c.call(check=True)
    c.check(out, lse)


def test_expanded_many_units_in_any_order():
    """More units than CTAs; max_k is only a hint; the same bits every time."""
    torch = _torch()
    rng = np.random.default_rng(95)
    news = rng.integers(0, 400, 30)
    c = Ragged(news, news + rng.integers(0, 100, 30), 16, 64, 32, 64, "bf16", 96)
    out, lse = c.call(check=True)
    c.check(out, lse)
    for max_k in (1, 1 << 30):
        o, l = c.call(max_k=max_k, check=True)
        assert torch.equal(_bits(o), _bits(out)) and torch.equal(l, lse)
    o, l = c.call(max_q=5000, check=True)
    assert torch.equal(_bits(o), _bits(out))


def test_expanded_strides_and_given_outputs():
    torch, fa = _torch(), _fa()
    c = Ragged([100, 150], [130, 150], 3, 96, 32, 80, "fp16", 97)
    T, Tk, H = 250, 280, 3

    def spread(x, pad):   # head-major memory with gaps
        y = torch.full((x.shape[1], x.shape[0] + 5, x.shape[2] + pad), math.nan, dtype=x.dtype, device="cuda")
        v = y[:, 3:3 + x.shape[0], pad // 2:pad // 2 + x.shape[2]].transpose(0, 1)
        v.copy_(x)
        return v
    q, k, v = spread(c.q, 16), spread(c.kv[..., :96], 32), spread(c.kv[..., 96:], 16)
    sh = torch.full((Tk, 48), math.nan, dtype=torch.float16, device="cuda")[:, 8:40]
    sh.copy_(c.shared)
    out = torch.full((T + 7, H, 96), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    o, l = fa.latent_attention_forward(q, k, sh, v, _i32(c.cu_q), _i32(c.cu_k), 150, 150, out=out[2:2 + T, :, 8:88], lse=lse, check=True)
    assert l is lse
    c.check(o, l)
    assert (out[:2] == 7).all() and (out[2 + T:] == 7).all() and (out[..., :8] == 7).all() and (out[..., 88:] == 7).all()
    # rows that are no request's, and keys that are nobody's
    out = torch.full((T, H, 80), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    fa.latent_attention_forward(q, k, sh, v, _i32(c.cu_q[1:]), _i32(c.cu_k[1:]), 150, 150, out=out, lse=lse, check=True)
    assert (out[:100] == 7).all() and (lse[:100] == 7).all()
    c.check(out, lse, rows=slice(100, None))


def test_expanded_bad_marks_are_reported():
    torch, fa = _torch(), _fa()
    c = Ragged([50, 60, 70], [50, 60, 70], 2, 64, 32, 64, "bf16", 98)
    for cq, ck in (([0, 50, 400, 180], c.cu_k), ([-5, 50, 110, 180], c.cu_k), (c.cu_q, [0, 50, 40, 180]), (c.cu_q, [0, 50, 110, 999])):
        out = torch.full((180, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        a = c.args()
        fa.latent_attention_forward(*a[:4], _i32(cq), _i32(ck), 70, 70, out=out)
        assert fa.fa_check_device_status(None) == fa.FA_ERR_INVALID_ARG
        _ok()
        good = [b for b in range(3) if 0 <= cq[b] <= cq[b + 1] <= 180 and cq[b + 1] - cq[b] <= 70 and 0 <= ck[b] <= ck[b + 1] <= 180]
        want = c.want()[0]
        for b in good:
            if (cq[b], cq[b + 1], ck[b], ck[b + 1]) == (c.cu_q[b], c.cu_q[b + 1], c.cu_k[b], c.cu_k[b + 1]):
                rows = slice(cq[b], cq[b + 1])
                assert np.abs(_f64(out[rows]) - want[rows]).max() < 0.1     # there at all; exactly: the other tests
    with pytest.raises(fa.FaError):
        c.call(max_q=60, check=True)     # a request of 70
    _ok()


def test_expanded_refusals_and_no_query():
    torch, fa = _torch(), _fa()
    c = Ragged([5, 6], [5, 6], 2, 64, 32, 64, "bf16", 99)
    q, k, sh, v, cq, ck = c.args()
    for args in ((q[..., :64], k, sh, v, cq, ck), (q, k[:, :1], sh, v, cq, ck), (q, k, sh[:5], v, cq, ck), (q, k, sh, v[:5], cq, ck), (q, k, sh, v, cq, ck[:2]),
                 (q, k, sh, v, cq.long(), ck), (q[0], k, sh, v, cq, ck)):
        with pytest.raises(ValueError):
            fa.latent_attention_forward(*args, 6, 6)
    with pytest.raises(TypeError):
        fa.latent_attention_forward(q, k.half(), sh, v, cq, ck, 6, 6)
    for kw in (dict(max_q=0), dict(max_k=0), dict(scale=-1.0)):
        with pytest.raises(fa.FaError):
            fa.latent_attention_forward(q, k, sh, v, cq, ck, **{**dict(max_q=6, max_k=6), **kw})
    out, lse = fa.latent_attention_forward(q[:0], k, sh, v, _i32([0, 0, 0]), ck, 0, 0, check=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, lse = fa.latent_attention_forward(q[:0], k[:0], sh[:0], v[:0], _i32([0]), _i32([0]), 0, 0, check=True)
    assert out.shape == (0, 2, 64)
    _ok()


# ------------------------------------------------------------ as they are used
def test_latent_serving_steps():
    """Prompts in the expanded form while their latents go into the cache, then drafts and single tokens in the absorbed
    form: tables, append and attention of two steps captured in a graph and replayed with new lengths, on a stream of their own."""
    torch, fa = _torch(), _fa()
    H, C, R, Dn, Dv, P, B = 4, 64, 32, 64, 48, 16, 3
    prompts, pages = np.array([37, 130, 16]), 20
    tab = lref.table(200, R)
    dev_tab = torch.from_numpy(tab).cuda()
    s = torch.cuda.Stream()
    cache = torch.full((pages, P, C + R), math.nan, dtype=torch.bfloat16, device="cuda")
    state = [_i32(np.zeros(B)), _i32(np.zeros((B, 10))), _i32(np.arange(pages)), _i32([pages])]   # lens, table, free, count

    def step(new, T, kv, qr, absorbed):
        lens, table, free, count = state
        slots, cu, after, left, _ = fa.kv_tables_step(new, lens, table, free, count, P, T)
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        row = (torch.searchsorted(cu, t, right=True, out_int32=True) - 1).clamp(max=B - 1).long()
        pos = torch.where(slots >= 0, lens[row] + t - cu[row], -1).int()
        turned = fa.latent_cache_append(kv[:, :C], kv[:, C:], slots, cache, qr, pos, dev_tab)
        out = lse = None
        if absorbed is not None:
            q = absorbed.clone()
            q[..., C:] = turned
            out, lse = fa.latent_paged_attention_forward(q, cache, table, after, C, cu, 3, scale=0.1)
        lens.copy_(after)
        count.copy_(left)
        return slots, cu, pos, turned, out, lse

    def turn(x, pos):
        return torch.from_numpy(lref.turn(x.float().cpu().numpy(), pos, tab, False)).to(torch.bfloat16).double().numpy()

    T0 = int(prompts.sum())
    kv0, q0 = _rand((T0, C + R), "bf16", 100).cuda(), _rand((T0, H, Dn + R), "bf16", 101).cuda()
    wk, wv = _rand((C, H * Dn), "bf16", 102, 0.1).cuda(), _rand((C, H * Dv), "bf16", 103, 0.1).cuda()
    k0, v0 = (kv0[:, :C] @ wk).view(T0, H, Dn), (kv0[:, :C] @ wv).view(T0, H, Dv)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        slots, cu, pos, turned, _, _ = step(_i32(prompts), T0, kv0, q0[..., Dn:], None)
        kr = cache.view(-1, C + R)[slots.long(), C:]
        full_q = torch.cat([q0[..., :Dn], turned], dim=-1)
        out, lse = fa.latent_attention_forward(full_q, k0, kr, v0, cu, cu, 130, 130)
    s.synchronize()
    _ok()
    p0 = np.concatenate([np.arange(n) for n in prompts])
    np.testing.assert_array_equal(pos.cpu().numpy(), p0)
    kr_want = turn(kv0[:, None, C:], p0)[:, 0]
    assert np.array_equal(_f64(kr), kr_want)
    latents = [np.concatenate([_f64(kv0[a:a + n, :C]), kr_want[a:a + n]], axis=1) for a, n in zip(np.cumsum(prompts) - prompts, prompts)]
    parts = []
    for a, n in zip(np.cumsum(prompts) - prompts, prompts):
        k = np.concatenate([_f64(k0[a:a + n]), np.broadcast_to(kr_want[a:a + n, None], (n, H, R))], axis=2)
        parts.append(lref.attend(_f64(full_q[a:a + n]), k, _f64(v0[a:a + n]), np.arange(n) + 1, 1 / math.sqrt(Dn + R)))
    lref.check(out, lse, [np.concatenate(x) for x in zip(*parts)], Dn + R, 130, np.abs(_f64(v0)).max(), torch.bfloat16)

    # two more steps, captured once and replayed three times
    news, T = [np.array([3, 1, 2]), np.array([1, 0, 1])], [8, 4]
    new_t = [_i32(n) for n in news]
    kv, qr = [torch.empty((t, C + R), dtype=torch.bfloat16, device="cuda") for t in T], [torch.empty((t, H, R), dtype=torch.bfloat16, device="cuda") for t in T]
    qa = [torch.empty((t, H, C + R), dtype=torch.bfloat16, device="cuda") for t in T]
    saved = [x.clone() for x in (*state, cache)]
    with torch.cuda.stream(s):
        for x in (*kv, *qr, *qa):
            x.zero_()
        for i in range(2):
            step(new_t[i], T[i], kv[i], qr[i], qa[i])
        for x, y in zip((*state, cache), saved):
            x.copy_(y)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = [step(new_t[i], T[i], kv[i], qr[i], qa[i]) for i in range(2)]
    lens = prompts.copy()
    for turn_no in range(3):
        for i in range(2):
            kv[i].copy_(_rand(kv[i].shape, "bf16", 110 + 10 * turn_no + i))
            qr[i].copy_(_rand(qr[i].shape, "bf16", 113 + 10 * turn_no + i))
            qa[i].copy_(_rand(qa[i].shape, "bf16", 116 + 10 * turn_no + i))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        _ok()
        for i in range(2):
            _, _, _, turned, out, lse = got[i]
            p = np.concatenate([np.arange(a, a + n) for a, n in zip(lens, news[i])])
            n_all = len(p)
            rows = np.concatenate([_f64(kv[i][:n_all, :C]), turn(kv[i][:n_all, None, C:], p)[:, 0]], axis=1)
            qs = np.concatenate([_f64(qa[i][:n_all, :, :C]), turn(qr[i][:n_all], p)], axis=2)
            parts, at = [], 0
            for b, n in enumerate(news[i]):
                latents[b] = np.concatenate([latents[b], rows[at:at + n]])
                lens[b] += n
                parts.append(lref.attend(qs[at:at + n], latents[b], latents[b][:, :C], lens[b] - n + 1 + np.arange(n), 0.1))
                at += n
            want = [np.concatenate(x) for x in zip(*parts)]
            top = max(np.abs(x).max() for x in latents)
            lref.check(out[:n_all], lse[:n_all], want, C + R, int(lens.max()), top, torch.bfloat16)


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own."""
    torch, fa = _torch(), _fa()
    cases = [Case([3000, 90], [1, 2], 64, 512, 64, 64, "bf16", 120), Case([2500, 10, 700], [1, 1, 1], 100, 256, 64, 16, "bf16", 121)]
    r = Ragged([400, 300], [500, 300], 8, 128, 64, 128, "bf16", 122)
    dev = [(c.q.cuda(), c.cache.cuda(), _i32(c.table), _i32(c.lens), c.C, _i32(c.cu), int(c.news.max())) for c in cases]
    ragged = r.args()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [fa.latent_paged_attention_forward(*d, scale=c.scale, stream=s) for d, c, s in zip(dev, cases, streams)]
        got.append(fa.latent_attention_forward(*ragged, 400, 500, stream=streams[2]))
    torch.cuda.synchronize()
    _ok()
    for c, (o, l) in zip(cases + [r], got):
        c.check(o, l)


def test_two_graphs_share_a_workspace():
    """Two graphs with the same workspace given, replayed one after the other."""
    torch, fa = _torch(), _fa()
    c = Case([3000, 900], [1, 1], 128, 512, 64, 64, "bf16", 123)
    d = (c.q.cuda(), c.cache.cuda(), _i32(c.table), _i32(c.lens), c.C, _i32(c.cu), 1)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 128), device="cuda")) for _ in range(2)]
    fa.latent_paged_attention_forward(*d, scale=c.scale, out=outs[0][0], lse=outs[0][1], workspace=ws, check=True)
    graphs = []
    for o, l in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.latent_paged_attention_forward(*d, scale=c.scale, out=o, lse=l, workspace=ws)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    _ok()
    for o, l in outs:
        c.check(o, l)


def test_expanded_a_long_request_among_many_short_ones():
    """Requests far shorter than the longest, fewer and more of them than one CTA counts."""
    torch = _torch()
    rng = np.random.default_rng(130)
    for B, H in ((300, 3), (2100, 1)):
        news = rng.integers(0, 4, B)
        news[B // 3] = 1500
        c = Ragged(news, news + rng.integers(0, 40, B) * (news > 0), H, 64, 32, 64, "bf16", 131)
        out, lse = c.call(check=True)
        c.check(out, lse)
        for _ in range(3):
            again = c.call()
            assert torch.equal(_bits(again[0]), _bits(out)) and torch.equal(again[1], lse)
    _ok()


def test_same_bits_while_the_memory_is_busy():
    """Loads that come late or early change nothing."""
    torch, fa = _torch(), _fa()
    c = Case([5000, 129, 64, 8000, 1, 3000], [1] * 6, 128, 512, 64, 64, "bf16", 132)
    d = (c.q.cuda(), c.cache.cuda(), _i32(c.table), _i32(c.lens), c.C, _i32(c.cu), 1)
    r = Ragged([700, 1, 900], [800, 60, 900], 8, 128, 64, 128, "fp16", 133)
    ragged = r.args()
    out, lse = fa.latent_paged_attention_forward(*d, scale=c.scale, check=True)
    c.check(out, lse)
    wide, wide_lse = fa.latent_attention_forward(*ragged, 900, 900, check=True)
    r.check(wide, wide_lse)
    side, x, y = torch.cuda.Stream(), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(side):
            y.copy_(x)
        o, l = fa.latent_paged_attention_forward(*d, scale=c.scale)
        w, m = fa.latent_attention_forward(*ragged, 900, 900)
        assert torch.equal(_bits(o), _bits(out)) and torch.equal(l, lse), i
        assert torch.equal(_bits(w), _bits(wide)) and torch.equal(m, wide_lse), i
    _ok()


@pytest.mark.parametrize("C,R", [(64, 0), (128, 0), (128, 64), (192, 64), (320, 64), (384, 128), (448, 128), (512, 0), (504, 72), (16, 560)])
def test_absorbed_widths(C, R):
    """Every number of 64-channel pieces, whole ones and cut ones, in pages of one box and of several."""
    for P in (16, 128):
        c = Case([300, 64, 5], [1, 2, 1], 24, C, R, P, "bf16", 134 + C)
        out, lse = c.call(check=True)
        c.check(out, lse)


@pytest.mark.parametrize("news,keys", [([260, 9], [300, 40]), ([300, 80], [360, 80]), ([300, 1], [500, 1]), ([700, 64], [801, 100]), ([513, 30], [513, 100])])
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_second_query_tile_beside_broken_values(news, keys, causal):
    """Requests of more than 256 rows, which two query tiles share, in front of one full of NaN and infinities: both tiles
    wait for a last tile's values and for the zeros behind them, also where loads come late."""
    torch, fa = _torch(), _fa()
    c = Ragged(news, keys, 5, 128, 64, 128, "bf16", 140)
    clean, clean_lse = c.call(causal=causal, check=True)
    c.check(clean, clean_lse, causal)
    a, n = c.cu_k[1], c.cu_q[1]
    c.kv[a::2], c.kv[a + 1::2], c.shared[a:] = math.nan, math.inf, math.nan
    broken = c.args()
    side, x, y = torch.cuda.Stream(), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(side):
            y.copy_(x)
        out, lse = fa.latent_attention_forward(*broken, max(news), max(keys), causal=causal)
        assert torch.equal(_bits(out[:n]), _bits(clean[:n])) and torch.equal(lse[:n], clean_lse[:n]), i
    _ok()


@pytest.mark.parametrize("lens,H", [([4096], 32), ([70001], 5), ([900], 128), ([3000] * 11, 32), ([2000, 1500, 300], 128)])
def test_absorbed_nan_through_the_join(lens, H):
    """A NaN in a query or in a cached row is a NaN in O and in the LSE, however many parts a request was cut into."""
    torch = _torch()
    c = Case(lens, [1] * len(lens), H, 128, 64, 64, "bf16", 142)
    clean, clean_lse = c.call(check=True)
    b, keep = len(lens) - 1, c.q.clone()
    c.q[b, H - 2, 5], c.q[0, 0, 150] = math.nan, math.nan
    out, lse = c.call(check=True)
    hit = torch.zeros(len(lens), H, dtype=torch.bool, device="cuda")
    hit[b, H - 2] = hit[0, 0] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(_bits(out[~hit]), _bits(clean[~hit])) and torch.equal(lse[~hit], clean_lse[~hit])
    for key, channel in ((0, 3), (lens[b] // 2, 180), (lens[b] - 1, 127)):
        c.q, was = keep, c.cache.clone()
        c.cache[c.table[b, key // c.P], key % c.P, channel] = math.nan
        out, lse = c.call(check=True)
        assert out[b].isnan().all() and lse[b].isnan().all(), (key, channel)
        assert torch.equal(_bits(out[:b]), _bits(clean[:b])) and torch.equal(lse[:b], clean_lse[:b])
        c.cache = was


@pytest.mark.parametrize("first", [0, 70, 3999])
def test_expanded_small_weights_in_fp16(first):
    """Many keys of 2^-25 to 2^-26 of the largest weight: together they are the output, whether the largest comes first or last.
    The weights enter the product times 2^7: below the type's normal range each is off by 2^-25 2^-7 of the largest at most, so
    what lref.tolerances says of such weights holds with a 2^-7th of the largest value."""
    torch = _torch()
    n, rows = 4000, 300
    c = Ragged([rows], [n], 2, 64, 32, 64, "fp16", 144)
    rng = np.random.default_rng(145)
    c.q[:], c.shared[:], c.kv[:] = 0, 0, 0
    c.q[..., 0], c.scale = 1, 1.0
    c.kv[..., 0] = torch.from_numpy(20 - math.log(2) * rng.uniform(25.1, 25.9, (n, 2))).half()
    c.kv[..., 64:] = torch.from_numpy(rng.uniform(8, 16, (n, 2, 64))).half()
    c.kv[first, :, 0], c.kv[first, :, 64:] = 20, 0
    out, lse = c.call(causal=False, scale=1.0, check=True)
    O, L, A, S = c.want(False)
    to, tl = lref.tolerances(O, L, A, S, 96, n, 16 * 2.0 ** -7, torch.float16)
    assert (O > 5e-4).all() and (to < 0.1 * O).all()
    assert (np.abs(_f64(out) - O) <= to).all(), np.abs(_f64(out) / O - 1).max()
    assert (np.abs(_f64(lse) - L) <= tl).all()


@pytest.mark.parametrize("dtype,inter", [("bf16", True), ("fp16", False)])
def test_latent_append_of_many_queries(dtype, inter):
    """Items enough (1.25 million) for two heads each, of an odd count; queries into views and in place."""
    torch, fa = _torch(), _fa()
    T, H, C, R, P = 2420, 129, 64, 64, 64
    rng = np.random.default_rng(146)
    slots = rng.permutation((-(-T // P) + 1) * P)[:T]
    slots[rng.random(T) < 0.05] = -1
    pos = np.where(rng.random(T) < 0.05, -1, rng.integers(0, 500, T))
    tab = lref.table(500, R)
    kv, q = _rand((T, C + R), dtype, 147).cuda(), _rand((T, H, C + R), dtype, 148).cuda()
    cache = _rand((-(-T // P) + 1, P, C + R), dtype, 149).cuda()
    want, on = cache.view(-1, C + R).clone(), slots >= 0
    k = torch.from_numpy(lref.turn(kv[:, None, C:].float().cpu().numpy(), pos, tab, inter)[:, 0]).to(_dt(dtype)).cuda()
    want[slots[on]] = torch.cat([kv[:, :C], k], dim=1)[torch.from_numpy(on).cuda()]
    wq = q.clone()
    wq[..., C:] = torch.from_numpy(lref.turn(q[..., C:].float().cpu().numpy(), pos, tab, inter)).to(_dt(dtype)).cuda()
    kw = dict(positions=_i32(pos), table=torch.from_numpy(tab).cuda(), interleaved=inter, check=True)
    out = fa.latent_cache_append(kv[:, :C], kv[:, C:], _i32(slots), cache, q_rope=q[..., C:], **kw)
    assert torch.equal(_bits(cache.view(-1, C + R)), _bits(want)) and torch.equal(_bits(out), _bits(wq[..., C:]))
    fa.latent_cache_append(kv[:, :C], kv[:, C:], _i32(slots), cache, q_rope=q[..., C:], q_out=q[..., C:], **kw)
    assert torch.equal(_bits(cache.view(-1, C + R)), _bits(want)) and torch.equal(_bits(q), _bits(wq))


@pytest.mark.parametrize("C,R,P", [(512, 64, 64), (64, 0, 128), (256, 32, 16)])
def test_absorbed_long_shares(C, R, P):
    """Shares of more than 16 tiles (ten requests of 17 thousand keys: 18 to each of 76 pairs)."""
    c = Case([17000 + 31 * i for i in range(10)], [1] * 10, 4, C, R, P, "bf16", 150)
    out, lse = c.call(check=True)
    c.check(out, lse)
