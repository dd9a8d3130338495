"""The row-by-row check of paged attention (tests/paged_rows.py): that it agrees with tests/paged_ref.py on
what the results are, that it passes their roundings, and that planted mistakes fail it, also in rows whose values are
small beside other rows' of the same cache."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests import paged_rows as rows

P = 16


def make(d, lens, news, Hk, G, seed, low, high):
    """A cache whose value scales are 2^low .. 2^(high - 1) by page and head, and queries of which one row is
    large, one tiny and one zero."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    need = -(-lens // P)
    cache = ref.Cache(int(need.sum()) + 3, Hk, P, d, seed)
    cache.scale["v"] = 2.0 ** rng.integers(low, high, cache.scale["v"].shape)
    cache.scale["k"] = 2.0 ** rng.integers(-12, -3, cache.scale["k"].shape)
    table, perm, at = np.full((len(lens), max(1, int(need.max()))), -1), rng.permutation(cache.pages), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(news)])
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), Hk * G, d))).bfloat16()
    q[0, 1] *= 50.0
    q[1 % len(q), 0] *= 1e-20
    q[2 % len(q), 2] = 0
    return cache, table, lens, cu, q


CASES = {d: dict(d=d, lens=[900, 30], news=[60, 40], Hk=2, G=2, seed=300 + d, low=-30, high=20) for d in (64, 128, 256)}


@pytest.fixture(scope="module", params=sorted(CASES))
def case(request):
    c = make(**CASES[request.param])
    cache, table, lens, cu, q = c
    d = q.shape[2]
    return c, d, rows.attend(cache, q.double().numpy(), table, lens, cu, 1 / math.sqrt(d), True)


def rounded(got, dtype):
    return torch.from_numpy(got[0]).to(dtype).double().numpy(), torch.from_numpy(got[1]).float().double().numpy()


def test_agrees_with_the_other_oracle(case):
    (cache, table, lens, cu, q), d, got = case
    want = ref.attend(cache, q.double().numpy(), table, lens, cu, 1 / math.sqrt(d), True)
    for a, b in zip(got, want):
        a, b = np.nan_to_num(a, neginf=-1.0), np.nan_to_num(b, neginf=-1.0)
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13 * np.abs(b).max())
    none = rows.attend(cache, q.double().numpy(), table, lens, cu, 0.3, False, [[[0, 2], [1]], [[1], [0]]])
    want = ref.attend(cache, q.double().numpy(), table, lens, cu, 0.3, False, [[[0, 2], [1]], [[1], [0]]])
    np.testing.assert_allclose(none[0], want[0], rtol=1e-12, atol=1e-13 * np.abs(want[0]).max())


def test_passes_the_rounded_result_and_sees_every_row(case):
    (cache, table, lens, cu, q), d, got = case
    assert rows.mismatch(*rounded(got, q.dtype), got, d, q.dtype) == []
    assert (rows.blind(got, d, q.dtype) > 0.5).mean() <= 0.01


def test_planted_mistakes_fail(case):
    (cache, table, lens, cu, q), d, got = case
    o, l = rounded(got, q.dtype)
    sees = np.isfinite(got[1])
    for h in range(4):
        for r in (slice(0, 60), slice(60, 100)):                       # one head of one request
            if not sees[r, h].any():
                continue
            for f in (0.0, 0.95, -1.0):
                bad = o.copy()
                bad[r, h] *= f
                assert rows.mismatch(bad, l, got, d, q.dtype), (h, r, f)
            bad = l.copy()
            bad[r, h] += 1e-2
            assert rows.mismatch(o, bad, got, d, q.dtype), (h, r)
    # keys whose values' scale is small left out of the sum
    big = {"k": cache.scale["k"], "v": cache.scale["v"]}
    small = big["v"] < 2.0 ** -20
    codes = cache.codes["k"].copy()
    cache.codes["k"][small] = 0
    off = rows.attend(cache, q.double().numpy(), table, lens, cu, 1 / math.sqrt(d), True)
    cache.codes["k"] = codes
    assert rows.mismatch(*rounded(off, q.dtype), got, d, q.dtype)
