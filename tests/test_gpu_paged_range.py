"""Attention over the paged cache at the ends of what its values may be."""

import numpy as np
import pytest

from oracle import paged_oracle as O
from test_gpu_paged import _attend_close, _dev, _f64, _ints

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
def test_large_and_small_values(ctx, dtype, d, size):
    """Values up to 2^114 / len and as far down, under scores that begin at a row's first and end just below 14 powers of 2 over it,
    where the weights are at their largest."""
    from cross_model_kv_amd import kvmap as K
    page, T = 64, 4000                                   # 2^100 * 1.99 * 4000 < 2^113
    n = -(-T // page)
    rng = np.random.default_rng(d)
    k, v = np.zeros((1, n, 1, page, d)), size * rng.uniform(-1.99, 1.99, (1, n, 1, page, d))
    k[..., 0] = np.where(np.arange(n * page).reshape(1, n, 1, page) < 128, 0.0, 9.625)      # nats: 13.9 powers of 2
    q = np.zeros((1, 1, 4, d))
    q[..., 0] = 1.0
    (kt, k64), (vt, v64), (qt, q64) = _dev(k, dtype), _dev(v, dtype), _dev(q, dtype)
    pages, lens = [list(range(n))], [T]
    for max_len in (T, n * page):
        out, lse = ctx.paged_attend(K.PagedCache(kt, vt), qt, _ints(pages), _ints(lens), max_len, scale=1.0, lse=True)
        torch.cuda.synchronize()
        ref = O.attend(dict(k=k64, v=v64), q64, pages, lens, 1.0)
        _attend_close(_f64(out), _f64(lse), ref, dtype, d, lens, False)
