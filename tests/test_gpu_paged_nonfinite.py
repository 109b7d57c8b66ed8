"""Attention over the paged cache with infinities and NaN in keys and values, with and without rotated queries: by whole sequences
and by pieces, with one tile of rows, with two, and with two blocks of them.  What is finite is held to test_gpu_paged.py's tolerances."""

import numpy as np
import pytest

from oracle import paged_oracle as O
from test_gpu_paged import THETA, _attend_close, _dev, _f64, _ints, _table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ODD = [np.inf, -np.inf, np.nan]


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


def _case(rng, lens, H, d, page):
    """A pool, its tables, and how to reach a sequence's token in it."""
    need = [-(-l // page) for l in lens]
    pages = _table(rng, sum(need) + 2, need, 5000 // page + 1)
    k, v = rng.standard_normal((2, 1, sum(need) + 2, H, page, d))
    return k, v, pages, lambda x, b, h, pos: x[0, pages[b][pos // page], h, pos % page]


def _run(ctx, k, v, q, pages, lens, dtype, d, rope, cut, scale=None):
    """What the call gives, the oracle's answer, and the oracle's with every key element finite (whose sums of |q k| bound scores)."""
    from cross_model_kv_amd import kvmap as K
    (kt, k64), (vt, v64), (qt, q64) = _dev(k, dtype), _dev(v, dtype), _dev(q, dtype)
    max_len = 5000 if cut else max(lens)
    rot = ctx.rope_table(max_len, d, theta=THETA) if rope else None
    r64 = None if rot is None else _f64(rot)[:max(lens)]
    out, lse = ctx.paged_attend(K.PagedCache(kt, vt), qt, _ints(pages), _ints(lens), max_len, rope=rot, lse=True, scale=scale)
    torch.cuda.synchronize()
    scale = d ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore"):
        ref = O.attend(dict(k=k64, v=v64), q64, pages, lens, scale, rot=r64)
        tame = O.attend(dict(k=np.where(np.isfinite(k64), k64, 0), v=v64), q64, pages, lens, scale, rot=r64)
    return _f64(out), _f64(lse), ref, tame


@pytest.mark.parametrize("cut", [False, True], ids=["own", "pieces"])
@pytest.mark.parametrize("rope", [False, True], ids=["plain", "turned"])
@pytest.mark.parametrize("n_q,G", [(1, 3), (4, 6), (16, 3)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
def test_keys(ctx, dtype, d, n_q, G, rope, cut):
    """A key with an element that is not finite, early in a sequence or among the last tokens that only some rows see.  An infinity
    gives a score of -infinity, which has no weight, or of +infinity, by the sign of the query's element: rows of both kinds."""
    lens, H, page = [40, 300, 640, 33, 700], 2, 16
    rng = np.random.default_rng([1, d, n_q, G])
    k, v, pages, at = _case(rng, lens, H, d, page)
    for b, l in enumerate(lens):
        for h in range(H):
            at(k, b, h, 5 if b % 2 else l - 1 - n_q // 2)[rng.integers(d)] = ODD[2] if b == 4 else ODD[(b + h) % 2]
    q = 1.5 * rng.standard_normal((len(lens), n_q, H * G, d))
    out, lse, ref, tame = _run(ctx, k, v, q, pages, lens, dtype, d, rope, cut)
    finite = np.isfinite(ref[0][:4]).all(-1)
    assert finite.any() and not finite.all()
    _attend_close(out, lse, (ref[0], ref[1], ref[2], tame[3]), dtype, d, lens, rope)


@pytest.mark.parametrize("cut", [False, True], ids=["own", "pieces"])
@pytest.mark.parametrize("rope", [False, True], ids=["plain", "turned"])
@pytest.mark.parametrize("n_q,G", [(5, 3), (8, 4), (16, 3), (16, 5)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
def test_values_that_later_rows_alone_see(ctx, dtype, d, n_q, G, rope, cut):
    """Drafted tokens with infinities and NaN in some dims of their values, and both in keys and values past a sequence's end: the rows
    that see a value have it, by its weight's sum, and no other row does.  (Such tiles are multiplied after the others, row by row, with
    the queries turned once more.)"""
    lens, H, page = [n_q, 100, 640, 33, 1], 2, 16
    rng = np.random.default_rng([2, d, n_q, G])
    k, v, pages, at = _case(rng, lens, H, d, page)
    used = sum((p[:-(-l // page)] for p, l in zip(pages, lens)), [])
    for x in (k, v):
        x[:, [i for i in range(x.shape[1]) if i not in used]] = np.nan
        for b, l in enumerate(lens):
            for pos in range(l, -(-l // page) * page):
                for h in range(H):
                    at(x, b, h, pos)[:] = ODD[pos % 3]
    for b, l in enumerate(lens[:4]):
        for h in range(H):
            for j in range(1 + h, min(n_q, l), 2):       # of tokens l - 1 - j, the last j + 1 rows see it
                at(v, b, h, l - 1 - j)[rng.choice(d, 6, replace=False)] = [np.nan, np.inf, -np.inf, np.inf, np.inf, -np.inf]
    q = 1.5 * rng.standard_normal((len(lens), n_q, H * G, d))
    out, lse, ref, tame = _run(ctx, k, v, q, pages, lens, dtype, d, rope, cut)
    fine = _attend_close(out, lse, ref, dtype, d, lens, rope)
    assert not fine[:4, -1].all() and fine[4].all() and not np.isnan(ref[1]).any()


@pytest.mark.parametrize("order", ["same tile", "other wave", "later step", "other piece", "before"])
@pytest.mark.parametrize("rope", [False, True], ids=["plain", "turned"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinity_far_below_the_largest_score(ctx, dtype, rope, order):
    """An infinite value whose score is 69 nats under the row's largest (a weight of 2^-99.5) stays one, wherever the two tokens lie;
    150 nats under, it is that or NaN, and nothing but its dim is touched."""
    from cross_model_kv_amd import kvmap as K
    d, page, T = 128, 16, 4600
    odd, high = {"same tile": (3, 20), "other wave": (3, 40), "later step": (3, 700), "other piece": (3, 4500), "before": (700, 3)}[order]
    rng = np.random.default_rng(3)
    for nats in (69.0, 150.0):
        k, v = np.zeros((1, T // page + 1, 1, page, d)), rng.standard_normal((1, T // page + 1, 1, page, d))
        k[0, high // page, 0, high % page, 0] = nats / 8
        v[0, odd // page, 0, odd % page, 7], v[0, odd // page, 0, odd % page, 9] = np.inf, -np.inf
        q = np.zeros((1, 1, 3, d))
        q[..., 0] = 8.0
        (kt, _), (vt, v64), (qt, _) = _dev(k, dtype), _dev(v, dtype), _dev(q, dtype)
        rot = None
        if rope:                                         # turns by nothing
            rot = torch.zeros((T, d // 2, 2), device="cuda")
            rot[..., 0] = 1.0
        out, lse = ctx.paged_attend(K.PagedCache(kt, vt), qt, _ints([list(range(T // page + 1))]), _ints([T]), T, scale=1.0, rope=rot,
                                    lse=True)
        torch.cuda.synchronize()
        out, lse = _f64(out), _f64(lse)
        seen = v64[0, high // page, 0, high % page]
        rest = [i for i in range(d) if i not in (7, 9)]
        # the other 4,599 tokens weigh e^-69 each; fp32's roundings of a score of 69 and one of the answer
        assert np.allclose(lse, nats, rtol=4 * 2.0 ** -24)
        assert (abs(out[..., rest] - seen[rest]) <= (2.0 ** -8 if dtype == "bf16" else 4 * 2.0 ** -24) * abs(seen[rest])).all()
        if nats < 76:
            assert (out[..., 7] == np.inf).all() and (out[..., 9] == -np.inf).all()
        else:
            assert not np.isfinite(out[..., [7, 9]]).any() and not (out[..., 7] == -np.inf).any() and not (out[..., 9] == np.inf).any()


@pytest.mark.parametrize("rope", [False, True], ids=["plain", "turned"])
@pytest.mark.parametrize("n_q,G", [(1, 3), (4, 6), (16, 3)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_queries(ctx, dtype, d, n_q, G, rope):
    """A query with an element that is not finite: its row is the formula's, or NaN where it is turned, and no other row is touched."""
    lens, H, page = [40, 300, 17], 2, 16
    rng = np.random.default_rng([4, d, n_q, G])
    k, v, pages, _ = _case(rng, lens, H, d, page)
    q = 1.5 * rng.standard_normal((len(lens), n_q, H * G, d))
    for b in range(len(lens)):
        q[b, n_q // 2, b, rng.integers(d)] = ODD[b]
    out, lse, ref, _ = _run(ctx, k, v, q, pages, lens, dtype, d, rope, False)
    tame = _run(ctx, k, v, np.where(np.isfinite(q), q, 0), pages, lens, dtype, d, rope, False)[2]
    r_out, r_lse = ref[0].copy(), ref[1].copy()
    if rope:
        for b in range(len(lens)):
            lost = np.isnan(out[b, n_q // 2, b]).any()
            assert lost == np.isnan(lse[b, n_q // 2, b])
            if lost:
                r_out[b, n_q // 2, b] = r_lse[b, n_q // 2, b] = np.nan
    _attend_close(out, lse, (r_out, r_lse, ref[2], tame[3]), dtype, d, lens, rope)
