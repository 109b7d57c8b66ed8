"""Writes of a few tokens, and small pages, on the GPU: every code and scale is the oracle's."""

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


def _write(ctx, K, rng, L, B, H, n, start, count, d, page, dtype, layout, spread=4.0):
    cnt = count if count is not None else [n] * B
    need = [max(-(-(s + m) // page), 1) for s, m in zip(start, cnt)]
    n_pages, max_pages = sum(need) + 2, max(need) + 1
    o = _pool(rng, L + 1, n_pages, H, page, d)
    c = _from_oracle(K, o)
    table = _table(rng, n_pages, need, max_pages)
    k, v, k64, v64 = _rows(rng, L, B, H, n, d, dtype, layout, spread)
    pages, st, ct = _ints(table), _ints(start), None if count is None else _ints(count)
    for again in range(2):
        ctx.q8_write(c, k, v, pages, st, count=ct, layer=1)
        if not again:
            assert Q.write(o, k64, v64, table, start, cnt, layer=1) == 0
        _same(c, o, f"write {again}")
    assert ctx.q8_dropped() == 0
    for dt in ("bf16", "f32"):
        gk, gv = ctx.q8_read(c, pages, st, n, count=ct, layer=1, n_layers=L, dtype=_dt(dt))
        rk, rv = Q.read(o, table, start, n, cnt, 1, L)
        np.testing.assert_array_equal(_f64(gk), rk)
        np.testing.assert_array_equal(_f64(gv), rv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_tokens_each_page_size(ctx, K, d, page, dtype):
    """One to nine tokens (where the choice of kernel changes), inside pages and over their ends, some sequences with fewer or
    none."""
    for n in (1, 2, 3, 7, 8, 9):
        rng = np.random.default_rng([2026, 861, d, page, n])
        start = [0, 1, page - 1, page, page + 3, 3 * page - n // 2]
        count = None if n % 2 else [n, n, 0, n - 1, n, n]
        _write(ctx, K, rng, 2, 6, 3, n, start, count, d, page, dtype, "tokens" if n % 3 else "heads")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 32), (128, 16), (128, 128)])
def test_long_writes_into_small_pages(ctx, K, d, page, dtype):
    rng = np.random.default_rng([2026, 862, d, page])
    _write(ctx, K, rng, 2, 3, 3, 201, [0, page - 5, 7], [201, 200, 0], d, page, dtype, "heads")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_tokens_out_of_the_ordinary(ctx, K, dtype):
    """Zeros, infinities, NaN and extremes among four new tokens beside older ones."""
    rng = np.random.default_rng([2026, 863])
    H, page, d, n, start = 6, 32, 128, 4, 5
    big = 3.38e38
    x = rng.standard_normal((2, 1, 1, H, n, d))
    x[:, :, :, 0] = 0.0
    x[:, :, :, 1, 0, 5] = np.nan
    x[:, :, :, 2, 1, 6], x[:, :, :, 2, 3, 7] = np.inf, -np.inf
    x[:, :, :, 3] *= big / 6
    x[:, :, :, 4] *= 1e-36
    x[:, :, :, 5] = np.nan
    o = _pool(rng, 1, 2, H, page, d)
    c = _from_oracle(K, o)
    k, v = (torch.from_numpy(y.astype(np.float32)).to(_dt(dtype)).cuda() for y in x)
    ctx.q8_write(c, k, v, _ints([[1]]), _ints([start]))
    Q.write(o, _f64(k), _f64(v), [[1]], [start], [n])
    _same(c, o)


def test_few_tokens_out_of_range_are_counted(ctx, K):
    rng = np.random.default_rng([2026, 864])
    H, n, page, d, n_pages = 2, 3, 16, 64, 8
    o = _pool(rng, 1, n_pages, H, page, d)
    c = _from_oracle(K, o)
    table = [[0, 1], [2, n_pages], [-1, 3], [4, 5], [6, 7]]
    start, count = [14, 14, 14, -1, 31], [3, 3, 3, 3, 3]
    k, v, k64, v64 = _rows(rng, 1, 5, H, n, d, "bf16", "heads")
    ctx.q8_write(c, k, v, _ints(table), _ints(start), count=_ints(count))
    want = Q.write(o, k64, v64, table, start, count)
    _same(c, o)
    assert ctx.q8_dropped() == want > 0


@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_up_to_a_small_page_of_tokens(ctx, K, d, page, dtype):
    """Ten to seventeen tokens, beginning at every place of a dword."""
    for n in (10, 12, 13, 15, 16, 17):
        rng = np.random.default_rng([2026, 865, d, page, n])
        start = [0, 1, 2, 3, page - 2, page + 5, 2 * page - n // 2]
        count = None if n % 2 else [n, n, n, n, n, 9, n - 3]
        _write(ctx, K, rng, 1, 7, 2, n, start, count, d, page, dtype, "heads" if n % 3 else "tokens")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages_that_begin_and_end_anywhere(ctx, K, d, page, dtype):
    """Writes longer than a small page whose first and last pages are partial, at every place of 16 bytes and of a dword."""
    for n in (18, 31, page + 1, 2 * page + 19):
        rng = np.random.default_rng([2026, 866, d, page, n])
        start = [0, 1, 6, 11, 15, page - 1, page + 7]
        count = [n, n, n - 1, n, n - 2, n, n // 2]
        _write(ctx, K, rng, 1, 7, 2, n, start, count, d, page, dtype, "heads")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("n", [1, 3, 8, 13])
def test_few_tokens_read_out_of_range(ctx, K, d, page, dtype, n):
    """Reads where pages, starts or counts are not what they have to be: NaN there, zeros past a count, the others whole."""
    rng = np.random.default_rng([2026, 867, d, n])
    H, n_pages, L = 2, 6, 2
    o = _pool(rng, L, n_pages, H, page, d)
    c = _from_oracle(K, o)
    table = [[0, 1], [2, n_pages], [-1, 3], [4, 5], [4, 5], [1, 0]]
    start = [page - 2, page - 1, page - n // 2, -1, 2 * page - 1, 3]
    for count in (None, [n, n - 1, n, n, n, n + 1]):
        ct = None if count is None else _ints(count)
        gk, gv = ctx.q8_read(c, _ints(table), _ints(start), n, count=ct, layer=0, n_layers=L, dtype=_dt(dtype))
        bad = [s < 0 or m > n for s, m in zip(start, count or [n] * 6)]
        want = Q.read(o, [t + [-1, -1] for t in table], [0 if x else s for x, s in zip(bad, start)], n,
                      [0 if x else m for x, m in zip(bad, count or [n] * 6)], 0, L)
        for got, ref in zip((gk, gv), want):
            ref[:, bad] = np.nan
            np.testing.assert_array_equal(_f64(got), ref)
