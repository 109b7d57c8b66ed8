"""The 8-bit paged cache on the GPU against the float64 oracle.

Writes and reads are exact: scales are powers of two, so a code is one correctly rounded value, and every
code and scale of the pool has to be the oracle's, the untouched ones included.

Attention, per output element, with w the softmax weights and A = sum_t w_t |v_t| of its row and dim:
  out itself is rounded once: u |ref|, u = 2^-8 (bf16) or 2^-24 (fp32), half a step relative;
  a weight is held in fp16 (2^-11 relative; two fp16 parts in an fp32 call, 2^-22), and an fp16 value
  below 2^-14 is off by up to 2^-25 of the scale it is held at, which is the largest w v_scale seen, or a
  code of 448: T 2^-25 448 max(w v_scale) (2^-36 for two parts);
  a score is a sum of d products in fp32 and two more roundings: delta = (d + 4) 2^-24 max_t scale sum |q k|,
  plus the rounding of exponents and statistics, 8 2^-24 (1 + |lse|); a weight's relative error is at most
  twice that, through itself and through the sum;
  the sums over tokens in fp32: T 2^-24 A at most.
The same delta and sum bound lse, with one rounding of its own value.
"""

import numpy as np
import pytest

from oracle import q8_oracle as Q

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


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _to_oracle(c):
    u = lambda t: t.view(torch.uint8).cpu().numpy().copy()
    return dict(k=u(c.k), v=u(c.v), ks=_f64(c.k_scale), vs=_f64(c.v_scale))


def _from_oracle(K, o, dtype_dev="cuda"):
    codes = lambda a: torch.from_numpy(a).to(dtype_dev).view(torch.float8_e4m3fn)
    sc = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype_dev)
    return K.Q8Cache(codes(o["k"]), codes(o["v"]), sc(o["ks"]), sc(o["vs"]))


def _same(c, o, where=""):
    g = _to_oracle(c)
    for name in ("ks", "vs", "k", "v"):
        bad = np.argwhere(~((g[name] == o[name]) | (np.isnan(g[name]) & np.isnan(o[name]))))
        assert not len(bad), f"{where} {name}: {len(bad)} differ, first at {bad[0]}: {g[name][tuple(bad[0])]} != {o[name][tuple(bad[0])]}"


def _pool(rng, L, n_pages, H, page, d, junk=True):
    """A pool that holds something everywhere, NaN codes among it."""
    o = Q.new_cache(L, n_pages, H, page, d)
    if junk:
        o["k"][:] = rng.integers(0, 256, o["k"].shape)
        o["v"][:] = rng.integers(0, 256, o["v"].shape)
        o["ks"][:] = 2.0 ** rng.integers(-12, -2, o["ks"].shape)
        o["vs"][:] = 2.0 ** rng.integers(-12, -2, o["vs"].shape)
    return o


def _table(rng, n_pages, need, max_pages):
    """Distinct pages for every sequence, the rest out of range."""
    ids = list(rng.permutation(n_pages))
    rows = []
    for u in need:
        rows.append([int(ids.pop()) for _ in range(u)] + [-7 if i % 2 else 1 << 29 for i in range(max_pages - u)])
    return rows


def _rounded(x, dtype):
    return torch.from_numpy(x.astype(np.float32)).to(_dt(dtype)).cuda()


# ---- write and read ----------------------------------------------------------------------

WRITES = [
    # L, B, H, n, start, count, d, page, dtype, layout
    (1, 1, 1, 1, [0], None, 128, 64, "bf16", "heads"),
    (1, 1, 8, 1, [1000], None, 128, 64, "bf16", "tokens"),
    (2, 3, 2, 1, [63, 64, 65], None, 64, 64, "bf16", "tokens"),
    (2, 3, 2, 1, [15, 16, 17], None, 64, 16, "f32", "heads"),
    (3, 1, 2, 64, [0], None, 128, 64, "bf16", "heads"),
    (1, 2, 3, 129, [0, 64], None, 128, 64, "bf16", "heads"),
    (1, 4, 2, 200, [0, 1, 63, 127], [200, 0, 1, 130], 128, 64, "bf16", "tokens"),
    (2, 3, 3, 77, [5, 31, 32], [77, 1, 33], 64, 32, "f32", "tokens"),
    (1, 2, 2, 300, [100, 3], [300, 299], 128, 128, "bf16", "heads"),
    (1, 2, 2, 300, [100, 3], [300, 299], 128, 128, "f32", "heads"),
    (1, 2, 5, 33, [16, 7], [33, 25], 64, 16, "bf16", "tokens"),
    (2, 1, 2, 65, [30], None, 64, 128, "f32", "heads"),
    (1, 2, 2, 49, [16, 15], None, 128, 16, "f32", "heads"),
    (1, 2, 2, 49, [16, 15], None, 128, 32, "f32", "heads"),
    (1, 2, 2, 49, [16, 15], None, 64, 64, "f32", "heads"),
    (1, 2, 2, 149, [16, 15], None, 128, 64, "f32", "heads"),
    (1, 2, 2, 49, [16, 15], None, 128, 16, "bf16", "heads"),
    (1, 2, 2, 149, [16, 15], None, 128, 32, "bf16", "heads"),
    (1, 2, 2, 149, [16, 15], None, 64, 32, "bf16", "heads"),
    (1, 2, 2, 300, [16, 15], None, 64, 128, "bf16", "heads"),
    (1, 2, 2, 300, [16, 15], None, 64, 64, "bf16", "heads"),
    (1, 2, 2, 49, [16, 15], None, 64, 16, "f32", "heads"),
]


def _rows(rng, L, B, H, n, d, dtype, layout, spread=4.0):
    """New rows as device views and as float64 arrays, of magnitudes that differ by page and head."""
    x = rng.standard_normal((2, L, B, H, n, d)) * np.exp(spread * rng.standard_normal((2, L, B, H, 1, 1)))
    if n > 1:
        x *= np.exp(spread * rng.standard_normal((2, L, B, H, n, 1)))
    if layout == "tokens":
        both = _rounded(np.concatenate([x[0], x[1]], 2).transpose(0, 1, 3, 2, 4).copy(), dtype)   # [L][B][n][2 H][d]
        k, v = both[:, :, :, :H].transpose(2, 3), both[:, :, :, H:].transpose(2, 3)
    else:
        k, v = _rounded(x[0], dtype), _rounded(x[1], dtype)
    return k, v, _f64(k), _f64(v)


@pytest.mark.parametrize("L,B,H,n,start,count,d,page,dtype,layout", WRITES)
def test_write_and_read_are_exact(ctx, K, L, B, H, n, start, count, d, page, dtype, layout):
    rng = np.random.default_rng([2026, 811, L, B, H, n, d, page])
    cnt = count if count is not None else [n] * B
    need = [-(-(s + m) // page) for s, m in zip(start, cnt)]
    n_pages, max_pages = sum(need) + 2, max(need) + 1
    o = _pool(rng, L + 1, n_pages, H, page, d)
    c = _from_oracle(K, o)
    table = _table(rng, n_pages, need, max_pages)
    k, v, k64, v64 = _rows(rng, L, B, H, n, d, dtype, layout)
    pages, st, ct = _ints(table), _ints(start), None if count is None else _ints(count)
    ctx.q8_write(c, k, v, pages, st, count=ct, layer=1)
    assert Q.write(o, k64, v64, table, start, cnt, layer=1) == 0
    _same(c, o, "once")
    ctx.q8_write(c, k, v, pages, st, count=ct, layer=1)     # the same again changes nothing
    _same(c, o, "twice")
    assert ctx.q8_dropped() == 0
    for dt in ("bf16", "f32"):
        gk, gv = ctx.q8_read(c, pages, st, n, count=ct, layer=1, n_layers=L, dtype=_dt(dt))
        rk, rv = Q.read(o, table, start, n, cnt, 1, L)
        np.testing.assert_array_equal(_f64(gk), rk)
        np.testing.assert_array_equal(_f64(gv), rv)


@pytest.mark.parametrize("dtype,page,d", [("bf16", 64, 128), ("f32", 16, 64), ("bf16", 128, 64)])
def test_tokens_written_one_by_one(ctx, K, dtype, page, d):
    """A sequence grows by one token a call; its scales grow with it, and earlier tokens are rounded again."""
    rng = np.random.default_rng([2026, 812, page, d])
    H, T = 2, page + 5
    o = Q.new_cache(1, 3, H, page, d)
    c = _from_oracle(K, o)
    table = [[2, 0, -1]]
    pages = _ints(table)
    grew = 0
    for t in range(T):
        x = rng.standard_normal((2, 1, 1, H, 1, d)) * (1.3 ** t if t % 3 else 1e-3)
        k, v = _rounded(x[0], dtype), _rounded(x[1], dtype)
        before = o["ks"].copy()
        ctx.q8_write(c, k, v, pages, _ints([t]))
        Q.write(o, _f64(k), _f64(v), table, [t], [1])
        grew += int((o["ks"] > before).any()) if t % page else 0
    assert grew > 5
    _same(c, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("start", [0, 3])
def test_values_out_of_the_ordinary(ctx, K, dtype, start):
    """Zeros, infinities, NaN, the type's extremes and its subnormals, in pages of their own and beside
    ordinary values; ties of the rounding."""
    rng = np.random.default_rng([2026, 813, start])
    H, page, d = 9, 16, 64
    big, tiny = (3.38e38, 9.2e-41) if dtype == "bf16" else (3.4e38, 1.4e-45)
    x = rng.standard_normal((2, 1, 1, H, page - start, d))
    x[:, :, :, 0] = 0.0
    x[:, :, :, 1, 0, 5] = np.nan
    x[:, :, :, 2, 1, 6] = np.inf
    x[:, :, :, 2, 1, 7] = -np.inf
    x[:, :, :, 3] *= big / 6
    x[:, :, :, 3, 0, 0] = -big
    x[:, :, :, 4] = tiny * rng.integers(-3, 4, x[:, :, :, 4].shape)
    x[:, :, :, 5] *= 1e-36
    x[:, :, :, 6] = np.nan
    x[:, :, :, 7] = rng.choice((Q._GRID[1:] + Q._GRID[:-1]) / 2, x[:, :, :, 7].shape)     # halfway between codes
    x[:, :, :, 7, 0, 0] = 448.0
    x[:, :, :, 8] = -0.0
    k, v = _rounded(x[0], dtype), _rounded(x[1], dtype)
    o = _pool(rng, 1, 2, H, page, d)
    c = _from_oracle(K, o)
    ctx.q8_write(c, k, v, _ints([[1]]), _ints([start]))
    Q.write(o, _f64(k), _f64(v), [[1]], [start], [page - start])
    _same(c, o)
    gk, gv = ctx.q8_read(c, _ints([[1]]), _ints([start]), page - start, dtype=torch.float32)
    rk, rv = Q.read(o, [[1]], [start], page - start, [page - start])
    np.testing.assert_array_equal(_f64(gk), rk)
    np.testing.assert_array_equal(_f64(gv), rv)


def test_read_into_parts_of_one_buffer(ctx, K):
    rng = np.random.default_rng([2026, 814])
    L, B, H, n, page, d = 2, 2, 3, 40, 32, 64
    o = _pool(rng, L, 6, H, page, d)
    o["k"] &= 0x77
    o["v"] &= 0x77
    c = _from_oracle(K, o)
    table = [[3, 0], [5, 1]]
    buf = torch.full((L, B, n, 2 * H + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = buf[:, :, :, :H].transpose(2, 3), buf[:, :, :, H:2 * H].transpose(2, 3)
    ctx.q8_read(c, _ints(table), _ints([1, 24]), n, count=_ints([40, 13]), out_k=k, out_v=v)
    rk, rv = Q.read(o, table, [1, 24], n, [40, 13], 0, L)
    np.testing.assert_array_equal(_f64(k), rk)
    np.testing.assert_array_equal(_f64(v), rv)
    assert (buf[:, :, :, 2 * H] == 7).all()


def test_what_is_out_of_range(ctx, K):
    """Bad starts, counts and pages: writes leave them out and count them, reads and attention answer NaN, and
    neither the other sequences nor the rest of the pool notice."""
    rng = np.random.default_rng([2026, 815])
    B, H, n, page, d, n_pages = 7, 2, 40, 16, 64, 12
    o = _pool(rng, 1, n_pages, H, page, d)
    o["k"] &= 0x77
    o["v"] &= 0x77
    c = _from_oracle(K, o)
    table = [[0, 1, 2], [3, n_pages, 4], [5, -1, 6], [7, 8, 9], [10, 11, 9], [0, 0, 0], [2147483647, -2147483648, 1]]
    start = [0, 0, 0, 20, -1, 0, 0]           # 3: its last tokens lie past the table; 4: a negative start
    count = [40, 40, 40, 40, 40, 41, 32]      # 5: more than n
    k, v, k64, v64 = _rows(rng, 1, B, H, n, d, "bf16", "heads")
    ctx.q8_write(c, k, v, _ints(table), _ints(start), count=_ints(count))
    want = Q.write(o, k64, v64, table, start, count)
    assert want == 2 * H * (1 + 1 + 1 + 1 + 1 + 2)
    _same(c, o)
    assert ctx.q8_dropped() == want
    assert ctx.q8_dropped() == 0
    gk, gv = ctx.q8_read(c, _ints(table), _ints(start), n, count=_ints(count), dtype=torch.float32)
    for b in range(B):
        bad = np.array([b in (4, 5) or not (0 <= t // page < 3 and 0 <= table[b][t // page] < n_pages)
                        for t in range(start[b], start[b] + n)])
        bad &= np.arange(n) < (n if b in (4, 5) else count[b])
        for g in (_f64(gk), _f64(gv)):
            np.testing.assert_array_equal(np.isnan(g[0, b]).all((0, 2)), bad)
            assert not np.isnan(g[0, b][:, ~bad]).any()
    lens = [40, 40, 15, 48, -1, 49, 0]
    q = torch.randn((B, 1, 2 * H, d), device="cuda")
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), 48, lse=True)
    for b, bad in enumerate([False, True, False, False, True, True, False]):
        assert bool(torch.isnan(out[b]).all()) == bad and bool(torch.isnan(out[b]).any()) == bad, b
        assert bool(torch.isnan(lse[b]).all()) == bad, b
    assert (out[6] == 0).all() and (lse[6] == -np.inf).all()


# ---- attention ----------------------------------------------------------------------------

def _check(out, lse, ref, T, d, dtype, where):
    ro, rl, f = ref
    u, w, floor = (2.0 ** -8, 2.0 ** -11, 2.0 ** -25) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22, 2.0 ** -36)
    empty = np.isneginf(rl)
    delta = (d + 4) * 2.0 ** -24 * f["abss"] + 8 * 2.0 ** -24 * (1 + np.where(empty, 0, np.abs(rl)))
    go, gl = _f64(out), _f64(lse)
    assert (go[empty] == 0).all() and np.isneginf(gl[empty]).all(), where
    bound = u * np.abs(ro) + (w + 2 * delta[..., None] + T * 2.0 ** -24) * f["absv"] + T * floor * 448 * f["wv"][..., None] + 1e-37
    err = np.abs(go - ro)
    worst = float((err / bound).max())
    lbound = delta + T * 2.0 ** -24 + 2.0 ** -24 * np.where(empty, 0, np.abs(rl))
    lworst = float((np.abs(gl[~empty] - rl[~empty]) / lbound[~empty]).max()) if (~empty).any() else 0.0
    print(f"[q8 attend] {where}: out err/bound {worst:.3f}, lse err/bound {lworst:.3f}", flush=True)
    assert np.isfinite(go).all() and worst <= 1.0, where
    assert lworst <= 1.0, where


def _held(rng, lens, H, page, d, L=1, layer=0, sharp=1.0):
    """An oracle cache that holds lens[b] tokens of every sequence; everything past them is junk, NaN codes among it."""
    need = [-(-t // page) for t in lens]
    n_pages, max_pages = sum(need) + 2, max(max(need), 1) + 1
    o = _pool(rng, L, n_pages, H, page, d)
    table = _table(rng, n_pages, need, max_pages)
    for b, t in enumerate(lens):
        if t:
            x = rng.standard_normal((2, 1, 1, H, t, d)) * np.exp(0.5 * rng.standard_normal((2, 1, 1, H, 1, d)))
            x[1] *= np.exp(rng.standard_normal((1, 1, H, t, 1)))
            Q.write(o, x[0] * sharp, x[1], [table[b]], [0], [t], layer)
    unused = set(range(n_pages)) - {p for r in table for p in r}
    for p in unused:
        o["ks"][:, p], o["vs"][:, p] = np.nan, np.inf
    return o, table


ATTENDS = [
    # lens, n_q, H, G, d, page, dtype
    ([1], 1, 1, 1, 128, 64, "bf16"),
    ([1], 1, 1, 1, 64, 16, "f32"),
    ([0, 1, 2, 3], 3, 2, 2, 64, 16, "bf16"),
    ([15, 16, 17, 0], 1, 2, 8, 128, 16, "bf16"),
    ([31, 32, 33, 64, 65], 1, 3, 5, 128, 32, "bf16"),
    ([63, 64, 65, 127, 128, 129], 2, 2, 4, 128, 64, "bf16"),
    ([255, 256, 257, 511], 1, 1, 16, 64, 128, "bf16"),
    ([255, 256, 257, 511], 1, 1, 16, 128, 128, "f32"),
    ([1000], 1, 2, 7, 128, 64, "bf16"),
    ([1000, 3], 1, 2, 3, 64, 32, "f32"),
    ([4097], 1, 1, 8, 128, 64, "bf16"),
    ([2049, 5, 0, 700], 4, 2, 5, 64, 16, "bf16"),
    ([300, 7, 0], 9, 2, 3, 128, 32, "f32"),
    ([333, 200, 5], 17, 2, 1, 128, 64, "bf16"),
    ([90, 40, 130], 64, 1, 3, 64, 64, "bf16"),
    ([200, 64, 65], 65, 2, 2, 128, 128, "bf16"),
    ([150], 150, 1, 5, 128, 64, "bf16"),
    ([257], 129, 1, 2, 64, 16, "f32"),
    ([70, 300], 70, 2, 3, 128, 32, "f32"),
    ([500], 33, 1, 24, 128, 64, "bf16"),
    ([130, 20], 1, 2, 40, 128, 64, "bf16"),
    ([600], 260, 1, 1, 128, 16, "bf16"),
    ([600], 300, 1, 1, 64, 32, "bf16"),
]


@pytest.mark.parametrize("lens,n_q,H,G,d,page,dtype", ATTENDS)
def test_attend_matches_oracle(ctx, K, lens, n_q, H, G, d, page, dtype):
    rng = np.random.default_rng([2026, 821, len(lens), max(lens), n_q, H, G, d, page])
    o, table = _held(rng, lens, H, page, d)
    c = _from_oracle(K, o)
    q = _rounded(1.5 * rng.standard_normal((len(lens), n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), max(max(lens), 1), lse=True)
    ref = Q.attend(o, _f64(q), table, lens, 0, d ** -0.5)
    _check(out, lse, ref, max(lens), d, dtype, f"lens {lens} n_q {n_q} H {H} G {G} d {d} page {page} {dtype}")
    again, lse2 = ctx.q8_attend(c, q, _ints(table), _ints(lens), max(max(lens), 1), lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert torch.equal(ctx.q8_attend(c, q, _ints(table), _ints(lens), max(max(lens), 1)), out)


def _random_attends(n=24):
    rng = np.random.default_rng([2026, 822])
    out = []
    for _ in range(n):
        B, n_q = int(rng.integers(1, 5)), int(rng.choice([1, 1, 2, 5, 16, 40, 100]))
        H, G = int(rng.integers(1, 4)), int(rng.integers(1, 13))
        top = int(np.exp(rng.uniform(0, np.log(60000 // (n_q * G * H + 20)))))
        lens = [int(rng.integers(0, top + 1)) for _ in range(B)]
        out.append((lens, n_q, H, G, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128])),
                    "f32" if rng.random() < 0.3 else "bf16"))
    return out


@pytest.mark.parametrize("lens,n_q,H,G,d,page,dtype", _random_attends())
def test_attend_random_cases(ctx, K, lens, n_q, H, G, d, page, dtype):
    """Seeded random lengths, queries, heads and pages, in the middle one of three layers, sharper scores, and a
    max_len far above the lengths."""
    rng = np.random.default_rng([2026, 823, max(lens), n_q, H, G, d, page])
    o, table = _held(rng, lens, H, page, d, L=3, layer=1, sharp=3.0)
    c = _from_oracle(K, o)
    table = [r + [-1] * 40 for r in table]
    q = _rounded(2 * rng.standard_normal((len(lens), n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), len(table[0]) * page, layer=1, scale=0.1, lse=True)
    ref = Q.attend(o, _f64(q), table, lens, 1, 0.1)
    _check(out, lse, ref, max(lens), d, dtype, f"lens {lens} n_q {n_q} H {H} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,G", [(1, 8), (4, 5), (40, 4)])
def test_scores_far_apart(ctx, K, dtype, n_q, G):
    """Scores that rise through the cache by hundreds, and pages whose value scales differ by 2^60: the running
    maximum moves all the time, and weights meet values of every size."""
    rng = np.random.default_rng([2026, 824, n_q, G])
    H, d, page, T = 2, 64, 16, 400
    o = Q.new_cache(1, 26, H, page, d)
    table = [list(range(25))]
    x = rng.standard_normal((2, 1, 1, H, T, d))
    x[0] += np.linspace(-30, 30, T)[:, None] * np.where(np.arange(H) % 2, -1, 1)[:, None, None] / 8
    x[1] *= 2.0 ** np.repeat(rng.integers(-30, 31, 25), page)[:, None]
    Q.write(o, x[0], x[1], table, [0], [T])
    c = _from_oracle(K, o)
    q = _rounded(1 + 0.2 * rng.standard_normal((1, n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints([T]), T, lse=True)
    _check(out, lse, Q.attend(o, _f64(q), table, [T], 0, d ** -0.5), T, d, dtype, f"far apart n_q {n_q} G {G} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,T,page", [(4, 37, 16), (4, 200, 64), (33, 100, 32), (150, 300, 64)])
def test_hidden_tokens_do_not_reach_a_row(ctx, K, dtype, n_q, T, page):
    """The newest tokens hold NaN and infinities; only the rows that see them become NaN, in the dims that hold one
    (keys: in all)."""
    rng = np.random.default_rng([2026, 825, n_q, T])
    H, G, d = 2, 3, 128
    o, table = _held(rng, [T], H, page, d)
    q = _rounded(rng.standard_normal((1, n_q, H * G, d)), dtype)
    clean = Q.attend(o, _f64(q), table, [T], 0, d ** -0.5)
    # head 0: values of token T - 2 in some dims; head 1: keys of token T - 3
    pv, pk = table[0][(T - 2) // page], table[0][(T - 3) // page]
    dims = [0, 5, 64, 127]
    o["v"][0, pv, 0, dims, (T - 2) % page] = [0x7F, 0xFF, 0x7F, 0xFF]
    o["k"][0, pk, 1, (T - 3) % page, 9] = 0xFF
    c = _from_oracle(K, o)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints([T]), T, lse=True)
    go, gl = _f64(out), _f64(lse)
    nan = np.zeros(go.shape, bool)
    nan[0, n_q - 2:, :G, dims] = True
    nan[0, max(n_q - 3, 0):, G:] = True
    np.testing.assert_array_equal(np.isnan(go), nan)
    np.testing.assert_array_equal(np.isnan(gl), nan[..., 1])
    ro, rl, f = clean
    keep = ~nan
    out[torch.from_numpy(nan).cuda()] = torch.from_numpy(ro).to(out)[torch.from_numpy(nan).cuda()]
    lse[torch.from_numpy(nan[..., 1]).cuda()] = torch.from_numpy(rl).to(lse)[torch.from_numpy(nan[..., 1]).cuda()]
    assert keep.any()
    _check(out, lse, clean, T, d, dtype, f"hidden n_q {n_q} T {T}")


def test_strided_queries_and_outputs(ctx, K):
    """q inside a projection's output, out inside a larger buffer, both in either order of heads and tokens."""
    rng = np.random.default_rng([2026, 826])
    lens, n_q, H, G, d, page = [70, 33], 5, 2, 3, 64, 32
    o, table = _held(rng, lens, H, page, d)
    c = _from_oracle(K, o)
    buf = _rounded(rng.standard_normal((2, n_q, H * G + 2 * H, d)), "bf16")
    q = buf[:, :, :H * G]
    want = Q.attend(o, _f64(q), table, lens, 0, d ** -0.5)
    res = torch.full((2, H * G, n_q + 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = res[:, :, 1:-1].transpose(1, 2)
    got, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), 70, out=out, lse=True)
    assert got is out
    _check(out, lse, want, 70, d, "bf16", "strided")
    assert (res[:, :, 0] == 3).all() and (res[:, :, -1] == 3).all()
    q2 = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ctx.q8_attend(c, q2, _ints(table), _ints(lens), 70), out)


def test_codes_past_4_gib(ctx, K):
    """Pages whose offsets pass 2^32 bytes: write, read and attend at both ends of a 5 GB pool."""
    rng = np.random.default_rng([2026, 827])
    H, page, d = 8, 128, 128
    n_pages = (5 << 30) // (H * page * d)
    c = ctx.q8_cache(1, n_pages, H, page, d)
    o = Q.new_cache(1, 4, H, page, d)
    small, table = [[1, 3], [0, 2]], [[n_pages - 1, 0], [1, n_pages - 2]]
    T = 200
    k, v, k64, v64 = _rows(rng, 1, 2, H, T, d, "bf16", "heads", spread=0.5)
    ctx.q8_write(c, k, v, _ints(table), _ints([0, 0]))
    Q.write(o, k64, v64, small, [0, 0], [T, T])
    gk, gv = ctx.q8_read(c, _ints(table), _ints([0, 0]), T)
    rk, rv = Q.read(o, small, [0, 0], T, [T, T])
    np.testing.assert_array_equal(_f64(gk), rk)
    np.testing.assert_array_equal(_f64(gv), rv)
    for n_q in (1, 40):
        q = _rounded(rng.standard_normal((2, n_q, H, d)), "bf16")
        out, lse = ctx.q8_attend(c, q, _ints(table), _ints([T, T]), T, lse=True)
        _check(out, lse, Q.attend(o, _f64(q), small, [T, T], 0, d ** -0.5), T, d, "bf16", f"past 4 GiB n_q {n_q}")
    del c
    torch.cuda.empty_cache()


def test_other_streams_and_graphs(ctx, K):
    """Decode steps (write, attend) on a side stream, and captured once and replayed while the sequences grow, each
    checked against the eager calls."""
    rng = np.random.default_rng([2026, 828])
    lens, H, G, d, page, steps = [60, 300], 2, 4, 128, 64, 6
    o, table = _held(rng, lens, H, page, d)
    need = -(-(max(lens) + steps) // page)
    extra = len(o["ks"][0])
    for key in ("k", "v", "ks", "vs"):
        o[key] = np.concatenate([o[key], np.zeros((1, 2 * need) + o[key].shape[2:], o[key].dtype)], 1)
    for b, r in enumerate(table):
        have = -(-lens[b] // page)
        table[b] = (r[:have] + list(range(extra + b * need, extra + (b + 1) * need)))[:need]
    eager, replayed = _from_oracle(K, o), _from_oracle(K, o)
    pages, max_len = _ints(table), need * page
    new = _rounded(rng.standard_normal((steps, 2, 2, H, 1, d)), "bf16")
    qs = _rounded(rng.standard_normal((steps, 2, 1, H * G, d)), "bf16")
    ctx.q8_reserve(eager, 2, 1, H * G, max_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = []
    with torch.cuda.stream(side):
        at = _ints(lens)
        for s in range(steps):
            ctx.q8_write(eager, new[s, 0], new[s, 1], pages, at)
            at = at + 1
            want.append(ctx.q8_attend(eager, qs[s], pages, at, max_len))
    torch.cuda.current_stream().wait_stream(side)
    kv, q, start, held = new[0].clone(), qs[0].clone(), _ints(lens), _ints(lens) + 1
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.q8_write(replayed, kv[0], kv[1], pages, start)
        ctx.q8_attend(replayed, q, pages, held, max_len, out=out)
    for s in range(steps):
        kv.copy_(new[s])
        q.copy_(qs[s])
        start.copy_(_ints(lens) + s)
        held.copy_(_ints(lens) + s + 1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[s]), s
    assert torch.equal(replayed.k.view(torch.uint8), eager.k.view(torch.uint8))
    assert torch.equal(replayed.v.view(torch.uint8), eager.v.view(torch.uint8))


def test_refusals_leave_outputs(ctx, K):
    c = ctx.q8_cache(2, 4, 2, 64, 128)
    pages, at = _ints([[0, 1], [2, 3]]), _ints([0, 0])
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    for over, status in [(dict(max_len=129), K.ERR_SHAPE), (dict(layer=2), K.ERR_SHAPE), (dict(scale=-1.0), K.ERR_INVALID_ARGUMENT)]:
        a = dict(max_len=128, out=out)
        a.update(over)
        with pytest.raises(K.KvmapError) as e:
            ctx.q8_attend(c, q, pages, at, **a)
        assert e.value.status == status
    with pytest.raises(K.KvmapError) as e:
        ctx.q8_attend(c, q, pages, at, 128, out=q)
    assert e.value.status == K.ERR_INVALID_ARGUMENT
    with pytest.raises(ValueError):
        ctx.q8_attend(c, q, pages.long(), at, 128, out=out)
    with pytest.raises(ValueError):
        ctx.q8_attend(c, q[..., :64], pages, at, 128)
    with pytest.raises(TypeError):
        ctx.q8_attend(c, q.half(), pages, at, 128)
    with pytest.raises(K.KvmapError) as e:
        ctx.q8_attend(c, q[:, :, :3], pages, at, 128)
    assert e.value.status == K.ERR_SHAPE
    k = torch.zeros((2, 2, 2, 3, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(K.KvmapError) as e:
        ctx.q8_write(c, k, k, pages, at, layer=1)
    assert e.value.status == K.ERR_SHAPE
    with pytest.raises(ValueError):
        ctx.q8_write(c, k, k[:1], pages, at)
    with pytest.raises(TypeError):
        ctx.q8_write(c, k, k.float(), pages, at)
    with pytest.raises(ValueError):
        ctx.q8_write(c, k, k, pages, _ints([0]))
    with pytest.raises(ValueError):
        ctx.q8_write(c, k.transpose(-1, -2), k.transpose(-1, -2), pages, at)
    with pytest.raises(K.KvmapError) as e:
        ctx.q8_read(c, pages, at, 3, out_k=k, out_v=k)
    assert e.value.status == K.ERR_INVALID_ARGUMENT
    torch.cuda.synchronize()
    assert (out == 5).all() and not c.k.view(torch.uint8).any() and not c.k_scale.any()
