"""The refusals of include/fa_rotary.h's and include/fa_latent.h's entry points, and the frequencies of rotary
positions, on the host.  As in test_abi.py the C calls pass fake addresses that are never dereferenced, so they run only
in a process that sees no GPU."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest

import online_softmax_tiling_gb300 as fa
from tests.test_abi import GPU_VISIBLE, ROOT
from tests.test_paged_abi import A, BAD, MISAL, UNSUP, _cache, lib  # noqa: F401 (lib: the fixture)

P = ctypes.addressof


def test_runs_where_no_gpu_is_visible():
    if not GPU_VISIBLE:
        pytest.skip("no GPU visible: the tests below run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", __file__],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


def _set(s, kw):
    for k, v in kw.items():
        if k.endswith("_stride") and isinstance(v, list):
            getattr(s, k)[:] = v
        else:
            setattr(s, k, v)
    return s


def _rot(**kw):
    return _set(fa.fa_rotary(A, A + 0x100, 100, 64, 0, 0), kw)


def _part(**kw):
    s = fa.fa_rotary_part(A + 0x1000, A + 0x2000)
    s.heads, s.x_stride[:], s.y_stride[:] = 4, [512, 128], [512, 128]
    return _set(s, kw)


ROTARY_REFUSALS = [(dict(table=None), BAD), (dict(positions=None), BAD), (dict(num_positions=0), BAD),
                   (dict(dim=0), UNSUP), (dict(dim=24), UNSUP), (dict(dim=528), UNSUP),
                   (dict(table=A + 4), MISAL), (dict(positions=A + 2), MISAL)]
PART_REFUSALS = [(dict(x=None), BAD), (dict(y=None), BAD), (dict(heads=0), BAD), (dict(x=A + 8), MISAL), (dict(y=A + 2), MISAL),
                 (dict(x_stride=[512, 0]), MISAL), (dict(x_stride=[-8, 128]), MISAL), (dict(y_stride=[512, 4]), MISAL),
                 (dict(y_stride=[1 << 40, 128]), MISAL)]


def _embed(lib, rot=None, q=None, k=None, T=5, d=128, dtype=1):  # noqa: F811
    rot, q = rot or _rot(), q or _part()
    return lib.fa_rotary_embed(P(rot), P(q), P(k) if k else None, T, d, dtype, None)


@pytest.mark.parametrize("kw,want", ROTARY_REFUSALS)
def test_rotary_refusals(lib, kw, want):  # noqa: F811
    assert _embed(lib, rot=_rot(**kw)) == want
    c, st = _cache(d=128), (ctypes.c_longlong * 2)(256, 128)
    rot = _rot(**kw)
    assert lib.fa_kv_cache_append_rotary(P(c), A, A, A, 5, P(st), P(st), P(rot), None, 1, None) == want


@pytest.mark.parametrize("kw,want", PART_REFUSALS)
def test_part_refusals(lib, kw, want):  # noqa: F811
    assert _embed(lib, q=_part(**kw)) == want
    assert _embed(lib, k=_part(**kw)) == want
    c, st, rot, q = _cache(d=128), (ctypes.c_longlong * 2)(256, 128), _rot(), _part(**kw)
    assert lib.fa_kv_cache_append_rotary(P(c), A, A, A, 5, P(st), P(st), P(rot), P(q), 1, None) == want
    l = _latents()
    assert lib.fa_latent_cache_append(P(l), A, 576, A, 576, A, 5, P(rot), P(q), 1, None) == want


@pytest.mark.parametrize("x,y,T,heads,want", [([512, 128], [512, 64], 5, 4, BAD), ([512, 128], [1024, 128], 5, 4, BAD),
                                              ([512, 128], [1024, 128], 5, 1, BAD), ([512, 128], [512, 64], 1, 4, BAD)])
def test_in_place_with_other_strides(lib, x, y, T, heads, want):  # noqa: F811
    q = _part(y=A + 0x1000, x_stride=x, y_stride=y, heads=heads)
    assert _embed(lib, q=q, T=T) == want and _embed(lib, k=q, T=T) == want
    assert _embed(lib, q=_part(y=A + 0x1000, x_stride=x, y_stride=y, heads=heads), T=0) == 0   # nothing is written


def test_rotary_call_refusals(lib):  # noqa: F811
    assert lib.fa_rotary_embed(None, P(_part()), None, 5, 128, 1, None) == BAD
    assert lib.fa_rotary_embed(P(_rot()), None, None, 5, 128, 1, None) == BAD
    assert _embed(lib, T=-1) == BAD
    assert _embed(lib, dtype=2) == BAD
    for d in (0, 8, 130, 520):
        assert _embed(lib, d=d) == UNSUP
    assert _embed(lib, rot=_rot(dim=64), d=48) == UNSUP              # more channels than the head has
    assert _embed(lib, q=_part(heads=1 << 20), T=1 << 20) == BAD     # items beyond 32 bits
    assert _embed(lib, T=0, q=_part(x=None, y=None), rot=_rot(table=None, positions=None)) == 0
    c, st, rot = _cache(d=128), (ctypes.c_longlong * 2)(256, 128), _rot(inverse=1)
    assert lib.fa_kv_cache_append_rotary(P(c), A, A, A, 5, P(st), P(st), P(rot), None, 1, None) == BAD
    assert lib.fa_kv_cache_append_rotary(P(c), A, A, A, 5, P(st), P(st), None, None, 1, None) == BAD
    assert lib.fa_kv_cache_append_rotary(P(c), A, A, A, 0, P(st), P(st), P(_rot()), None, 1, None) == 0


def _latents(**kw):
    return _set(fa.fa_latent_cache(A, 10, 16, 512, 64), kw)


LATENT_CACHE_REFUSALS = [(dict(rows=None), BAD), (dict(num_pages=0), BAD), (dict(page_size=8), BAD), (dict(page_size=256), BAD),
                         (dict(value_dim=0), UNSUP), (dict(value_dim=520, rope_dim=0), UNSUP), (dict(value_dim=100), UNSUP),
                         (dict(rope_dim=-8), UNSUP), (dict(rope_dim=12), UNSUP), (dict(rope_dim=72), UNSUP),
                         (dict(num_pages=1 << 28), BAD), (dict(rows=A + 8), MISAL)]


@pytest.mark.parametrize("kw,want", LATENT_CACHE_REFUSALS)
def test_latent_cache_refusals(lib, kw, want):  # noqa: F811
    c = _latents(**kw)
    assert lib.fa_latent_cache_append(P(c), A, 576, A, 576, A, 5, None, None, 1, None) == want
    assert lib.fa_latent_paged_fwd(P(_paged(cache=c))) == want
    assert lib.fa_latent_paged_workspace_size(P(_paged(cache=c))) == 0


def test_latent_append_refusals(lib):  # noqa: F811
    def call(cache=None, latent=A, ls=576, rope=A, rs=576, slots=A, T=5, rot=None, q=None, dtype=1):
        return lib.fa_latent_cache_append(P(cache or _latents()), latent, ls, rope, rs, slots, T, P(rot) if rot else None,
                                          P(q) if q else None, dtype, None)
    assert call(latent=None) == BAD and call(rope=None) == BAD and call(slots=None) == BAD
    assert call(T=-1) == BAD and call(dtype=5) == BAD and call(T=(1 << 30) + 1) == BAD
    assert call(q=_part()) == BAD                       # queries without a table
    assert call(rot=_rot(dim=48)) == BAD and call(rot=_rot(inverse=1)) == BAD
    assert call(ls=0) == MISAL and call(rs=4) == MISAL and call(latent=A + 8) == MISAL and call(slots=A + 2) == MISAL
    assert call(T=0, latent=None, rope=None, slots=None) == 0
    assert lib.fa_latent_cache_append(None, A, 576, A, 576, A, 5, None, None, 1, None) == BAD


def _paged(**kw):
    a = fa.fa_latent_paged_args()
    a.q, a.o, a.lse, a.block_table, a.lens = A, A + 0x100, A + 0x200, A + 0x300, A + 0x400
    a.cache = kw.pop("cache", None) or _latents()
    a.q_stride[:], a.o_stride[:] = [576 * 4, 576], [512 * 4, 512]
    a.T = a.B = 3
    a.H, a.max_q, a.max_pages, a.scale, a.causal, a.dtype = 4, 1, 20, 0.1, 1, fa.FA_BF16
    return _set(a, kw)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(block_table=None), BAD), (dict(lens=None), BAD),
    (dict(B=0), BAD), (dict(T=-1), BAD), (dict(H=0), BAD), (dict(max_q=0), BAD), (dict(max_pages=0), BAD), (dict(T=4), BAD),
    (dict(max_q=2), BAD), (dict(scale=0.0), BAD), (dict(scale=math.nan), BAD), (dict(dtype=2), BAD),
    (dict(max_pages=1 << 27), BAD), (dict(T=16385, B=16385), UNSUP), (dict(cu_q=A, max_q=1 << 30), BAD),
    (dict(T=16384, B=16384, max_pages=1 << 25), BAD),   # tiles beyond 32 bits
    (dict(q=A + 8), MISAL), (dict(o=A + 8), MISAL), (dict(lse=A + 2), MISAL), (dict(cu_q=A + 2), MISAL),
    (dict(q_stride=[2304, 4]), MISAL), (dict(o_stride=[0, 512]), MISAL),
    (dict(workspace=None), BAD), (dict(workspace=A + 16, workspace_bytes=1 << 40), MISAL), (dict(workspace=A, workspace_bytes=100), BAD)])
def test_latent_paged_refusals(lib, kw, want):  # noqa: F811
    assert lib.fa_latent_paged_fwd(P(_paged(**kw))) == want


def test_latent_paged_without_a_query(lib):  # noqa: F811
    for kw in (dict(T=0, B=0), dict(T=0, cu_q=A), dict(T=0, B=0, block_table=None, lens=None, max_q=0), dict(T=0, cu_q=A, q=None, o=None, lse=None)):
        assert lib.fa_latent_paged_fwd(P(_paged(**kw))) == 0
        assert lib.fa_latent_paged_workspace_size(P(_paged(**kw))) == 0
    assert lib.fa_latent_paged_fwd(None) == BAD


def _full(**kw):
    a = fa.fa_latent_args()
    a.q, a.k, a.k_rope, a.v, a.o, a.lse, a.cu_q, a.cu_k = (A + 0x100 * i for i in range(8))
    a.q_stride[:], a.k_stride[:], a.v_stride[:], a.o_stride[:], a.k_rope_stride = [768, 192], [1024, 256], [1024, 256], [512, 128], 64
    a.T, a.Tk, a.B, a.H, a.Dn, a.R, a.Dv, a.max_q, a.max_k, a.scale, a.causal, a.dtype = 30, 50, 2, 4, 128, 64, 128, 20, 30, 0.1, 1, 0
    return _set(a, kw)


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, BAD) for n in ("q", "k", "k_rope", "v", "o", "lse", "cu_q", "cu_k")],
    (dict(B=0), BAD), (dict(T=-1), BAD), (dict(Tk=-1), BAD), (dict(H=0), BAD), (dict(max_q=0), BAD), (dict(max_k=0), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=math.inf), BAD), (dict(dtype=3), BAD),
    (dict(Dn=0), UNSUP), (dict(Dn=136), UNSUP), (dict(Dn=60), UNSUP), (dict(R=0), UNSUP), (dict(R=72), UNSUP), (dict(Dv=4), UNSUP),
    (dict(Dv=136), UNSUP), (dict(T=(1 << 30) + 1), BAD), (dict(H=1 << 22, max_q=1 << 20), BAD),
    (dict(q=A + 8), MISAL), (dict(v=A + 4), MISAL), (dict(lse=A + 1), MISAL), (dict(cu_k=A + 2), MISAL),
    (dict(k_stride=[1024, 0]), MISAL), (dict(v_stride=[1020, 256]), MISAL), (dict(k_rope_stride=0), MISAL)])
def test_latent_refusals(lib, kw, want):  # noqa: F811
    assert lib.fa_latent_fwd(P(_full(**kw))) == want


def test_latent_without_a_query(lib):  # noqa: F811
    for kw in (dict(T=0), dict(T=0, B=0, cu_q=None, cu_k=None), dict(T=0, q=None, k=None, k_rope=None, v=None, o=None, lse=None, max_q=0, max_k=0)):
        assert lib.fa_latent_fwd(P(_full(**kw))) == 0
    assert lib.fa_latent_fwd(None) == BAD


def test_tensors_must_be_on_a_cuda_device():
    torch = pytest.importorskip("torch")
    x, i, t = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 64)
    for f, args in ((fa.rotary_embed, (x, x, i, t)), (fa.kv_cache_append_rotary, (x, x, x, i, t, i, x, x, t, t)),
                    (fa.latent_cache_append, (x[:, 0], x[:, 0], i, x)), (fa.latent_attention_forward, (x, x, x, x, i, i, 1, 1))):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(ValueError):
        fa.latent_paged_attention_forward(x, x, x, i, 8, scale=0.1)
    with pytest.raises(TypeError):
        fa.rotary_embed(None, x, i, t)


# ------------------------------------------------- frequencies and tables
def test_frequencies():
    pytest.importorskip("torch")
    w, f = fa.rotary_frequencies(8)
    np.testing.assert_allclose(w.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    assert f == 1.0
    w, f = fa.rotary_frequencies(8, scaling="linear", factor=4.0)
    np.testing.assert_allclose(w.numpy(), [0.25, 0.025, 0.0025, 0.00025], rtol=1e-15)
    w, f = fa.rotary_frequencies(8, scaling="base", factor=16.0)
    np.testing.assert_allclose(w.numpy()[[0, 3]], [1.0, 0.001 / 16], rtol=1e-14)   # the slowest pair alone is divided by 16


@pytest.mark.parametrize("dim,factor,length", [(64, 40.0, 4096), (128, 8.0, 8192), (16, 2.0, 100)])
def test_frequencies_by_bands(dim, factor, length):
    pytest.importorskip("torch")
    w, f = fa.rotary_frequencies(dim, scaling="bands", factor=factor, original_length=length)
    plain = 10000.0 ** (-2.0 * np.arange(dim // 2) / dim)
    turns = length * plain / (2 * math.pi)
    ratio = w.numpy() / plain
    eps = 2.0 ** -50   # two powers, each off by a step or so (2^-52), and the mixing
    assert (np.diff(ratio) <= eps).all() and (ratio <= 1 + eps).all() and (ratio >= 1 / factor - eps).all()
    # a pair's width outside of the two limits nothing is mixed any more
    step = 10000.0 ** (2.0 / dim)
    np.testing.assert_allclose(ratio[turns > 32 * step], 1.0, rtol=eps)
    np.testing.assert_allclose(ratio[turns < 1 / step], 1 / factor, rtol=1e-14)
    inside = (turns < 32 / step) & (turns > step)
    assert ((ratio < 1 - eps) & (ratio > 1 / factor + eps))[inside].all() and inside.any()
    assert f == pytest.approx(0.1 * math.log(factor) + 1)


def test_table_far_positions():
    torch = pytest.importorskip("torch")
    w, _ = fa.rotary_frequencies(32)
    t = fa.rotary_table(200001, w, factor=1.5, device="cpu").numpy()
    assert t.shape == (200001, 32) and t.dtype == np.float32
    for p in (0, 1, 65537, 200000):
        a = np.asarray([math.fmod(p * x, 2 * math.pi) for x in w.tolist()])
        # angles up to 2e5 in 64 bits: off by 2^-52 of that at most twice; then the rounding to fp32
        tol = 2e5 * 2.0 ** -51 + 1.5 * 2.0 ** -24
        assert np.abs(t[p, :16] - 1.5 * np.cos(a)).max() <= tol and np.abs(t[p, 16:] - 1.5 * np.sin(a)).max() <= tol
    assert torch.equal(fa.rotary_table(3, w, device="cpu"), fa.rotary_table(9, w, device="cpu")[:3])


def test_frequency_refusals():
    pytest.importorskip("torch")
    for kw in (dict(dim=7), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, base=math.inf), dict(dim=8, scaling="linear", factor=0.5),
               dict(dim=8, scaling="other"), dict(dim=8, scaling="bands", factor=2.0), dict(dim=2, scaling="base", factor=2.0),
               dict(dim=8, scaling="bands", factor=2.0, original_length=100, fast_turns=1.0)):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(**kw)
    with pytest.raises(ValueError):
        fa.rotary_table(0, fa.rotary_frequencies(8)[0], device="cpu")
