"""Writes and reads of 9 to 16 tokens of many pages, which a wave takes with its rows in registers, on the GPU: every code and scale of
the pool is the oracle's, and every value read is scale times code."""

import os
import re

import numpy as np
import pytest

from oracle import q8_oracle as Q
from test_gpu_q8 import _dt, _f64, _from_oracle, _ints, _pool, _rows, _same, _table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def K():
    from cross_model_kv_amd import kvmap as K
    return K


@pytest.fixture(scope="module")
def ctx(K):
    c = K.Context(0)
    yield c
    c.close()


def _limits():
    """The limits that choose the kernel, as its source has them: the most tokens of the smaller one and of this one, pages."""
    from cross_model_kv_amd import build
    src = open(os.path.join(build.CSRC, "q8_pages.hip")).read()
    few, some = map(int, re.search(r"kFew = (\d+), kSome = (\d+);", src).groups())
    return few, some, int(re.search(r"kManyPages = (\d+);", src)[1])


def _by_waves(dtype, d, page, read):
    """Pages that the general kernel would take by workgroups: those that a wave of that one cannot hold."""
    parts = page * d * (2 if dtype == "bf16" else 4) // 16
    return parts > (256 if read and dtype == "bf16" else 512)


L, B, H = 10, 16, 8
STARTS = [0, 1, 2, 3, 5, 6, 9, 14]


def _shapes():
    return [(dt, d, p) for dt in ("bf16", "f32") for d in (64, 128) for p in (16, 32, 64, 128)
            if _by_waves(dt, d, p, False) or _by_waves(dt, d, p, True)]


@pytest.mark.parametrize("dtype,d,page", _shapes())
@pytest.mark.parametrize("n", [9, 11, 14, 16])
def test_some_tokens_of_many_pages(ctx, K, dtype, d, page, n):
    """Starts at every place of a dword and of 16 bytes, over the ends of pages, and sequences with fewer tokens or none."""
    few, some, many = _limits()
    pages_of = (n + 2 * page - 2) // page * B * H * L * 2
    assert few < n <= some and pages_of >= many
    rng = np.random.default_rng([2026, 891, d, page, n])
    start = [s for s in STARTS] + [page - 1, page - 2, page - 7, page - n // 2, page, 2 * page - 9, page + 3, 2 * page - 16]
    count = [n, n, n, n, n, n, n, n, n, n, n, n, 0, n - 1, 1, 8]
    rng.shuffle(count)
    need = [max(-(-(s + m) // page), 1) for s, m in zip(start, count)]
    n_pages, max_pages = sum(need) + 2, max(need) + 1
    o = _pool(rng, L, n_pages, H, page, d)
    c = _from_oracle(K, o)
    table = _table(rng, n_pages, need, max_pages)
    k, v, k64, v64 = _rows(rng, L, B, H, n, d, dtype, "tokens" if n % 2 else "heads")
    pages, st, ct = _ints(table), _ints(start), _ints(count)
    ctx.q8_write(c, k, v, pages, st, count=ct)
    assert Q.write(o, k64, v64, table, start, count) == 0
    _same(c, o, "once")
    ctx.q8_write(c, k, v, pages, st, count=ct)
    _same(c, o, "twice")
    assert ctx.q8_dropped() == 0
    rk, rv = Q.read(o, table, start, n, count, 0, L)
    for dt in ("bf16", "f32"):
        gk, gv = ctx.q8_read(c, pages, st, n, count=ct, dtype=_dt(dt))
        np.testing.assert_array_equal(_f64(gk), rk)
        np.testing.assert_array_equal(_f64(gv), rv)


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 64), ("f32", 64, 128)])
def test_some_tokens_out_of_range(ctx, K, dtype, d, page):
    """Bad starts, counts and pages among many: left out and counted, NaN when read, and the others whole."""
    few, some, many = _limits()
    n = 13
    assert few < n <= some and (n + 2 * page - 2) // page * B * H * L * 2 >= many
    rng = np.random.default_rng([2026, 892, d])
    start = [page - 5] * B
    count = [n] * B
    table = [[2 * b, 2 * b + 1] for b in range(B)]
    start[1], count[2], count[3], start[4] = -1, n + 1, -2, 2 * page - 3
    table[5][0], table[6][1], table[7] = -1, 2 * B, [2147483647, -2147483648]
    o = _pool(rng, L, 2 * B, H, page, d)
    o["k"] &= 0x77
    o["v"] &= 0x77
    c = _from_oracle(K, o)
    k, v, k64, v64 = _rows(rng, L, B, H, n, d, dtype, "heads")
    ctx.q8_write(c, k, v, _ints(table), _ints(start), count=_ints(count))
    want = Q.write(o, k64, v64, table, start, count)
    _same(c, o)
    assert ctx.q8_dropped() == want > 0
    gk, gv = ctx.q8_read(c, _ints(table), _ints(start), n, count=_ints(count), dtype=_dt(dtype))
    bad = [b in (1, 2, 3) for b in range(B)]
    rk, rv = Q.read(o, [t + [-1] for t in table], [0 if x else s for x, s in zip(bad, start)], n, [0 if x else n for x in bad], 0, L)
    for got, ref in ((gk, rk), (gv, rv)):
        ref[:, bad] = np.nan
        np.testing.assert_array_equal(_f64(got), ref)
