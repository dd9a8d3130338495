"""Paged attention on the GPU against 64 bits with a tolerance of each row's own (tests/paged_rows.py)."""
import math

import pytest

from tests import paged_rows as rows
from tests import test_gpu_paged as base
from tests.test_paged_rows import P, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from online_softmax_tiling_gb300 import build
    build.build()
    yield


_ok = base._ok


# ------------------------------------------------- value scales far apart, row by row
def _same(case, out, lse, scale, causal=True, selected=None, log2_top=6):
    cache, table, lens, cu, q = case
    got = rows.attend(cache, q.double().numpy(), table, lens, cu, scale, causal, selected)
    assert (rows.blind(got, q.shape[2], q.dtype, log2_top) > 0.5).sum() <= 1   # (the row of large queries, d = 256)
    rows.check(out, lse, got, q.shape[2], q.dtype, log2_top)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 2, 3, 8])
@pytest.mark.parametrize("news", [[60, 40], [8, 3], [1, 1]])
def test_rows_of_small_values_keep_their_precision(d, splits, news):
    """Prompts, drafts and single tokens over pages whose value scales differ by 2^50: every row is held to its
    own size."""
    case = make(d, [900, 40], news, 2, 2, 310 + d + news[0], -30, 20)
    out, lse = base._attend(*case, news, num_splits=splits)
    _ok()
    _same(case, out, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 2, 3, 16])
@pytest.mark.parametrize("news", [[60, 40], [1, 1]])
def test_value_scales_as_far_apart_as_documented(d, splits, news):
    """Scales from 2^-60 (a page of zeros) to 2^36, the widest range whose sums are promised."""
    case = make(d, [900, 40], news, 2, 2, 330 + d + news[0], -60, 37)
    out, lse = base._attend(*case, news, num_splits=splits)
    _ok()
    _same(case, out, lse, 1 / math.sqrt(d), log2_top=8)


@pytest.mark.parametrize("low,high,top", [(-30, 20, 6), (-60, 37, 8)])
@pytest.mark.parametrize("d,G", [(64, 4), (128, 4), (128, 16), (256, 8)])
def test_equal_shares_over_a_wide_range_of_scales(d, G, low, high, top):
    lens = [900, 20, 0, 333] * 8
    case = make(d, lens, [1] * len(lens), 1, G, 350 + d + G, low, high)
    wide = base._wide_table(case[1], P, 456 * 66 * 32 // len(lens))
    out, lse = base._attend(case[0], wide, *case[2:], [1])
    _ok()
    _same(case, out, lse, 1 / math.sqrt(d), log2_top=top)
