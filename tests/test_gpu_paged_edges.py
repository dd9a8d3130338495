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
