"""The paged cache in the model's own type on the GPU against the float64 oracle.

Appends and reads move values and unrotated keys bit for bit, and leave everything else in the pool as it was.  A rotated
element is x c - y s from fp32 tables: one rounding of a product and one of the sum in fp32, each 2^-24 of at most
|x c| + |y s|, and the rounding to the cache's type, u |ref| with u = 2^-8 (bf16) or 2^-24 (fp32), half a step relative.
(The last two are one and the same in fp32, which leaves room; below 2^-126 a step is 2^-149, and bf16's 2^-133.)

Attention, per output element, with w the softmax weights and A = sum_t w_t |v_t| of its row and dim:
  out itself is rounded once: u |ref|;
  a bf16 call's weight is two bf16 parts, the second one's rounding 2^-8 of at most 2^-8: 2^-16 A;
  a score is a sum of d products in fp32, of a query turned in fp32 (2 roundings an element) and held in 24 bits or
  more (1), with two more roundings: delta = (d + 6) 2^-24 max_t scale sum |q k|, plus the rounding of exponents and
  statistics, 8 2^-24 (1 + |lse|); a weight's relative error is at most twice that, through itself and through the sum;
  a turned query's element is off by what |x c| + |y s| is: the sum |q k| is taken of a query sqrt 2 as large;
  the sums over tokens in fp32: T 2^-24 A at most.
The same delta and sum bound lse, with one rounding of its own value.
"""

import numpy as np
import pytest

from oracle import paged_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

THETA = 1.0e6


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


def _u(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _bits(t):
    return t.detach().contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


def _dev(x, dtype):
    """(device tensor, the float64 values that it holds)"""
    t = torch.from_numpy(np.ascontiguousarray(x).astype(np.float32)).to(_dt(dtype))
    return t.cuda(), t.float().double().numpy()


def _pool(K, rng, L, n_pages, H, page, d, dtype, odd=True):
    """A pool that holds something everywhere, infinities and NaN among it; the cache and its values."""
    shape = (L, n_pages, H, page, d)
    x = rng.standard_normal((2,) + shape)
    if odd:
        for val in (np.nan, np.inf, -np.inf):
            x[rng.random(x.shape) < 0.002] = val
    (k, k64), (v, v64) = _dev(x[0], dtype), _dev(x[1], dtype)
    return K.PagedCache(k, v), dict(k=k64, v=v64)


def _table(rng, n_pages, need, max_pages):
    """Distinct pages for every sequence, the rest out of range."""
    ids = list(rng.permutation(n_pages))
    return [[int(ids.pop()) for _ in range(u)] + [-7 if i % 2 else 1 << 29 for i in range(max_pages - u)] for u in need]


def _rows(rng, L, B, H, n, d, dtype, layout):
    """Keys and values [L][B][H][n][d] in a layout, and their values."""
    x = rng.standard_normal((L, B, n, 2 * H, d))
    both, b64 = _dev(x, dtype)
    if layout == "tokens":
        k, v = both[:, :, :, :H].transpose(2, 3), both[:, :, :, H:].transpose(2, 3)
    else:
        k, v = both[:, :, :, :H].transpose(2, 3).contiguous(), both[:, :, :, H:].transpose(2, 3).contiguous()
    return k, v, b64[:, :, :, :H].transpose(0, 1, 3, 2, 4), b64[:, :, :, H:].transpose(0, 1, 3, 2, 4)


def _turned_close(got, ref, size, dtype, where):
    tol = _u(dtype) * abs(ref) + 2 * 2.0 ** -24 * size + 2.0 ** -133
    bad = np.argwhere(~(abs(got - ref) <= tol))
    assert not len(bad), f"{where}: {len(bad)} off, first at {bad[0]}: {got[tuple(bad[0])]} for {ref[tuple(bad[0])]}"


ROWS = [
    # L, B, H, n, start, count, d, page, dtype, layout, rope
    (1, 1, 1, 1, [0], None, 128, 64, "bf16", "heads", True),
    (1, 1, 8, 1, [1000], None, 128, 64, "bf16", "tokens", True),
    (2, 3, 2, 1, [63, 64, 65], None, 64, 64, "bf16", "tokens", False),
    (2, 3, 2, 1, [15, 16, 17], None, 64, 16, "f32", "heads", True),
    (3, 1, 2, 64, [0], None, 128, 64, "bf16", "heads", False),
    (1, 2, 3, 129, [0, 64], None, 128, 64, "bf16", "heads", True),
    (1, 4, 2, 200, [0, 1, 63, 127], [200, 0, 1, 130], 128, 64, "bf16", "tokens", True),
    (2, 3, 3, 77, [5, 31, 32], [77, 1, 33], 64, 32, "f32", "tokens", True),
    (1, 2, 2, 300, [100, 3], [300, 299], 128, 128, "f32", "heads", True),
    (7, 1, 5, 33, [16], None, 128, 16, "bf16", "heads", True),
    (2, 1, 2, 65, [30], None, 64, 128, "f32", "heads", False),
    (9, 2, 1, 3, [14, 200], None, 64, 16, "bf16", "tokens", True),
]


@pytest.mark.parametrize("case", range(len(ROWS)))
def test_append_and_read(K, ctx, case):
    L, B, H, n, start, count, d, page, dtype, layout, rope = ROWS[case]
    rng = np.random.default_rng([11, case])
    need = [-(-(s + (n if count is None else count[b])) // page) for b, s in enumerate(start)]
    n_pages, max_pages = sum(need) + 3, max(max(need), 1) + 1
    cache, o = _pool(K, rng, L + 1, n_pages, H, page, d, dtype)
    pages = _table(rng, n_pages, need, max_pages)
    k, v, k64, v64 = _rows(rng, L, B, H, n, d, dtype, layout)
    rot = ctx.rope_table(max(start) + n, d, theta=THETA) if rope else None
    rot64 = _f64(rot) if rope else None
    before = {x: _bits(getattr(cache, x)).copy() for x in "kv"}
    print(f"[paged rows] case {case}", flush=True)
    cnt = None if count is None else _ints(count)
    for _ in range(2):    # appending the same tokens again changes nothing
        ctx.paged_append(cache, k, v, _ints(pages), _ints(start), count=cnt, layer=1, rope=rot)
    torch.cuda.synchronize()
    dropped, size = O.append(o, k64, v64, pages, start, count, layer=1, rot=rot64)
    assert dropped == 0 and ctx.paged_dropped() == 0
    touched = np.zeros(o["k"].shape, bool)
    for at in O.places(o, pages, start, count, n).values():
        if at not in (None, "past"):
            touched[1:1 + L, at[0], :, at[1]] = True
    for x in "kv":
        assert np.array_equal(_bits(getattr(cache, x))[~touched], before[x][~touched]), f"{x}: what is not appended to changed"
    assert np.array_equal(_f64(cache.v)[touched], o["v"][touched])
    if rope:
        _turned_close(_f64(cache.k)[touched], o["k"][touched], size[touched], dtype, "keys")
    else:
        assert np.array_equal(_f64(cache.k)[touched], o["k"][touched])

    # reading back what the cache holds now, as it is and stripped, into rows of either layout
    held = dict(k=_f64(cache.k), v=_f64(cache.v))
    for strip in (None, rot):
        if layout == "tokens":
            buf = torch.full((L, B, n, 2 * H, d), 7.0, dtype=_dt(dtype), device="cuda")
            out = dict(out_k=buf[:, :, :, :H].transpose(2, 3), out_v=buf[:, :, :, H:].transpose(2, 3))
        else:
            out = {}
        gk, gv = ctx.paged_read(cache, _ints(pages), _ints(start), n, count=cnt, layer=1, n_layers=L, rope=strip, **out)
        torch.cuda.synchronize()
        rk, rv, rs = O.read(held, pages, start, n, count, layer=1, n_layers=L, rot=None if strip is None else rot64)
        assert np.array_equal(_f64(gv), rv)
        if strip is None:
            assert np.array_equal(_f64(gk), rk)
        else:
            _turned_close(_f64(gk), rk, rs, dtype, "stripped keys")


def test_tables(ctx):
    """Cosines and sines are float64's rounded to fp32 (half a step, 2^-24, of at most 1; the angles' own rounding in float64 is
    2^-53 of up to 10^6)."""
    for d, kw in ((128, dict(theta=1.0e4)), (64, dict(theta=5.0e5)), (64, dict(inv_freq=[0.5 / (i + 1) for i in range(32)]))):
        for pos0 in (0, 130000):
            got = _f64(ctx.rope_table(777, d, pos0=pos0, **kw))
            ref = O.table(777, d, pos0=pos0, **kw)
            assert abs(got - ref).max() <= 2.0 ** -25 + 2.0 ** -32


def test_far_positions(K, ctx):
    """A key appended at position 131,071 by its table's last row."""
    rng = np.random.default_rng(5)
    d, page, pos = 128, 64, 131071
    cache, o = _pool(K, rng, 1, 2, 2, page, d, "f32", odd=False)
    pages = [[-1] * (pos // page) + [1]]
    rot = ctx.rope_table(pos + 1, d, theta=1.0e4)
    k, v, k64, v64 = _rows(rng, 1, 1, 2, 1, d, "f32", "heads")
    ctx.paged_append(cache, k, v, _ints(pages), _ints([pos]), rope=rot)
    exact = O.table(1, d, theta=1.0e4, pos0=pos)[0]
    ref, size = O.turn(k64[0, 0, :, 0], exact), O.turn_size(k64[0, 0, :, 0], exact)
    # the table's own rounding: half a step of fp32 of either factor
    assert (abs(_f64(cache.k)[0, 1, :, pos % page] - ref) <= 2.0 ** -24 * abs(ref) + 3 * 2.0 ** -24 * size).all()


def test_out_of_range_tokens_are_left_out(K, ctx):
    """Bad starts, counts, pages, positions past the page table and past the rotations: nothing of them is written, all are
    counted, and reading them gives NaN."""
    rng = np.random.default_rng(6)
    L, H, n, d, page = 2, 3, 40, 64, 16
    start = [0, -1, 5, 3, 60, 20, 2 ** 31 - 30, 0]
    count = [40, 40, 41, -1, 40, 30, 40, 7]
    pages = [[0, 99, 1, -1, 2], [3] * 5, [4] * 5, [5] * 5, [6, 6, 6, 7, 8], [9, 10, 11, 12, 13], [14] * 5, [15, 16, -1, -1, -1]]
    cache, o = _pool(K, rng, L, 20, H, page, d, "bf16", odd=False)
    k, v, k64, v64 = _rows(rng, L, len(start), H, n, d, "bf16", "heads")
    rot = ctx.rope_table(70, d, theta=1.0e4)
    before = _bits(cache.k).copy()
    ctx.paged_dropped()
    ctx.paged_append(cache, k, v, _ints(pages), _ints(start), count=_ints(count), rope=rot)
    torch.cuda.synchronize()
    dropped, size = O.append(o, k64, v64, pages, start, count, rot=_f64(rot))
    assert dropped == ctx.paged_dropped() and ctx.paged_dropped() == 0 and dropped > 100
    touched = size != 0
    assert np.array_equal(_bits(cache.k)[~touched], before[~touched])
    assert np.array_equal(_f64(cache.v), o["v"])
    _turned_close(_f64(cache.k), o["k"], size, "bf16", "keys")
    for strip in (None, rot):
        gk, gv = ctx.paged_read(cache, _ints(pages), _ints(start), n, count=_ints(count), rope=strip)
        torch.cuda.synchronize()
        held = dict(k=_f64(cache.k), v=_f64(cache.v))
        rk, rv, rs = O.read(held, pages, start, n, count, rot=None if strip is None else _f64(rot))
        assert np.array_equal(np.isnan(_f64(gv)), np.isnan(rv)) and np.isnan(rv).any()
        assert np.array_equal(np.isnan(_f64(gk)), np.isnan(rk))
        ok = ~np.isnan(rk)
        assert np.array_equal(_f64(gv)[ok], rv[ok])
        _turned_close(_f64(gk)[ok], rk[ok], rs[ok], "bf16", "keys")


# ---- attention -----------------------------------------------------------------------------

ATTEND = [
    # B, n_q, H, G, lens, d, page, dtype, rope
    (1, 1, 1, 1, [1], 128, 64, "bf16", True),
    (1, 1, 8, 2, [130], 128, 64, "bf16", True),
    (3, 1, 2, 8, [0, 1, 700], 128, 64, "bf16", False),
    (4, 1, 3, 3, [0, 709, 513, 31], 128, 32, "f32", True),
    (2, 1, 2, 16, [129, 640], 64, 16, "bf16", True),
    (2, 1, 2, 17, [129, 640], 128, 16, "bf16", True),
    (1, 1, 2, 33, [300], 128, 64, "bf16", False),
    (1, 1, 1, 40, [300], 64, 128, "f32", False),
    (2, 1, 2, 20, [1500, 33], 128, 64, "f32", True),
    (3, 4, 4, 5, [2, 1201, 63], 64, 16, "bf16", True),
    (3, 4, 4, 5, [2, 1201, 63], 64, 16, "f32", False),
    (2, 16, 2, 3, [15, 530], 128, 64, "bf16", True),
    (2, 16, 1, 8, [700, 16], 128, 32, "bf16", False),
    (2, 7, 3, 1, [1, 129], 128, 128, "f32", True),
    (70, 1, 1, 2, [(37 * i) % 400 for i in range(70)], 64, 16, "bf16", True),
    (70, 2, 1, 2, [(37 * i) % 900 for i in range(70)], 128, 32, "bf16", False),
]


def _attend_case(K, ctx, seed, B, n_q, H, G, lens, d, page, dtype, rope, spread=1.5, odd=False, max_len=None):
    rng = np.random.default_rng(seed)
    need = [-(-l // page) for l in lens]
    n_pages, max_pages = sum(need) + 2, max(max(need), 1) + 1
    cache, o = _pool(K, rng, 2, n_pages, H, page, d, dtype, odd=odd)
    pages = _table(rng, n_pages, need, max_pages)
    q, q64 = _dev(spread * rng.standard_normal((B, n_q, H * G, d)), dtype)
    rot = ctx.rope_table(max(max(lens), 1), d, theta=THETA) if rope else None
    max_len = max(lens) if max_len is None else max_len
    return cache, o, pages, q, q64, rot, max_len


def _attend_close(out, lse, ref, dtype, d, lens, rope, where=""):
    r_out, r_lse, size, prod = ref
    u, T = _u(dtype), max(max(lens), 1)
    with np.errstate(invalid="ignore"):
        delta = (d + 6) * 2.0 ** -24 * prod * (2 ** 0.5 if rope else 1) + 8 * 2.0 ** -24 * (1 + np.where(np.isfinite(r_lse), abs(r_lse), 0))
        weights = 2.0 ** -16 if dtype == "bf16" else 0.0
        tol = u * abs(r_out) + (weights + 2 * delta[..., None] + T * 2.0 ** -24) * size + 2.0 ** -133
        ltol = delta + T * 2.0 ** -24 + 2.0 ** -24 * abs(r_lse)
        fine = np.isfinite(r_out)
        same = np.where(fine, abs(out - r_out) <= tol, (out == r_out) | (np.isnan(out) & np.isnan(r_out)))
        bad = np.argwhere(~same)
        assert not len(bad), f"{where} out: {len(bad)} off, first at {bad[0]}: {out[tuple(bad[0])]} for {r_out[tuple(bad[0])]}, tolerance {tol[tuple(bad[0])]}"
        same = np.where(np.isfinite(r_lse), abs(lse - r_lse) <= ltol, (lse == r_lse) | (np.isnan(lse) & np.isnan(r_lse)))
        bad = np.argwhere(~same)
        assert not len(bad), f"{where} lse: {len(bad)} off, first at {bad[0]}: {lse[tuple(bad[0])]} for {r_lse[tuple(bad[0])]}"
    return fine


@pytest.mark.parametrize("cut", [False, True], ids=["own", "long"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(K, ctx, case, cut):
    """Every case by whole sequences where they are short enough, and (max_len far past them) by pieces."""
    B, n_q, H, G, lens, d, page, dtype, rope = ATTEND[case]
    cache, o, pages, q, q64, rot, max_len = _attend_case(K, ctx, [21, case], *ATTEND[case])
    if cut:
        wide = -(-5000 // page)
        pages = [p + [-1] * (wide - len(p)) for p in pages]
        max_len = 5000
        rot = ctx.rope_table(5000, d, theta=THETA) if rope else None
    print(f"[paged attend] case {case} cut {cut}", flush=True)
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, layer=1, rope=rot, lse=True)
    again, lse2 = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, layer=1, rope=rot, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    ref = O.attend(o, q64, pages, lens, d ** -0.5, layer=1, rot=None if rot is None else _f64(rot))
    _attend_close(_f64(out), _f64(lse), ref, dtype, d, lens, rope)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("n_q", [1, 5, 16])
def test_what_a_row_does_not_see(K, ctx, dtype, d, n_q):
    """NaN and infinities in every token past a sequence's end and, for drafted tokens, in tokens that only later rows
    see: they reach the rows that see them, as the formula has it, and no other."""
    page, H, G = 16, 2, 3
    lens = [n_q, 100, 640, 33]
    cache, o, pages, q, q64, rot, max_len = _attend_case(K, ctx, [31, n_q, d], len(lens), n_q, H, G, lens, d, page, dtype, False)
    rng = np.random.default_rng(8)
    for x in "kv":
        t = _f64(getattr(cache, x))
        for b, l in enumerate(lens):
            for pos in range(l, -(-l // page) * page):
                t[:, pages[b][pos // page], :, pos % page] = [np.nan, np.inf, -np.inf][pos % 3]
        t[:, [i for i in range(t.shape[1]) if i not in sum(pages, [])]] = np.nan
        for b, l in enumerate(lens):
            for j in range(1, n_q):          # values alone: a key that is not finite hides the values' behaviour
                if x == "v" and b < 3 and j % 2:
                    pos = l - j
                    if pos >= 0:
                        dims = rng.choice(d, 6, replace=False)
                        t[:, pages[b][pos // page], :, pos % page, dims] = np.array([np.nan, np.inf, -np.inf, np.inf, np.inf, -np.inf])[:, None, None]
        if x == "k" and n_q > 1:
            t[:, pages[3][(lens[3] - 1) // page], :, (lens[3] - 1) % page, 3] = np.nan
        new, n64 = _dev(t, dtype)
        getattr(cache, x).copy_(new)
        o[x] = n64
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, layer=1, lse=True)
    torch.cuda.synchronize()
    ref = O.attend(o, q64, pages, lens, d ** -0.5, layer=1)
    fine = _attend_close(_f64(out), _f64(lse), ref, dtype, d, lens, False)
    assert fine.all() == (n_q == 1)


def test_lost_pages_and_bad_lengths(K, ctx):
    """A row that sees a token of a page out of range is NaN, and so is a sequence whose length is out of range; the others
    are not touched."""
    for dtype, page in (("bf16", 16), ("f32", 64)):
        B, n_q, H, G, d = 6, 3, 2, 2, 64
        lens = [200, 200, 66, 40, 40, 90]
        cache, o, pages, q, q64, rot, _ = _attend_case(K, ctx, [41, page], B, n_q, H, G, lens, d, page, dtype, True)
        pages[1][5 * 16 // page] = 1 << 29       # in the middle
        pages[2][64 // page] = -3                # tokens 64, 65: seen by the last two rows alone
        given = list(lens)
        given[3], given[4] = -1, 201
        out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(given), 200, layer=0, rope=rot, lse=True)
        torch.cuda.synchronize()
        r = O.attend(o, q64, pages, lens, d ** -0.5, layer=0, rot=_f64(rot))
        for x in r[:2]:
            x[3:5] = np.nan
        assert np.isnan(r[1][1]).all() and np.isnan(r[1][2, 1:]).all() and not np.isnan(r[1][2, 0]).any()
        _attend_close(_f64(out), _f64(lse), r, dtype, d, lens, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_whose_weight_adds_nothing(K, ctx, dtype):
    """A first token with nearly all of a row's weight and values of zero: the answer is made of the small weights."""
    B, n_q, H, G, d, page, lens = 2, 1, 2, 4, 128, 64, [900, 2300]
    cache, o, pages, q, q64, rot, max_len = _attend_case(K, ctx, [51], B, n_q, H, G, lens, d, page, dtype, False, spread=0.5)
    for b in range(B):
        for x, val in (("k", None), ("v", 0.0)):
            t = getattr(cache, x)
            for h in range(H):
                # along the mean query of the heads that share it, long enough for scores of 15 to 30 nats
                at = (0, pages[b][0], h, 0)
                t[at] = val if val is not None else (q[b, 0, h * G:(h + 1) * G].float().mean(0) * 40).to(t.dtype)
    o = dict(k=_f64(cache.k), v=_f64(cache.v))
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, lse=True)
    torch.cuda.synchronize()
    ref = O.attend(o, q64, pages, lens, d ** -0.5)
    _attend_close(_f64(out), _f64(lse), ref, dtype, d, lens, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_rise_and_fall(K, ctx, dtype):
    """Scores that grow by hundreds over a sequence, and that start at their largest: the running maximum moves, or never."""
    B, n_q, H, G, d, page, lens = 2, 1, 1, 2, 64, 32, [1500, 1500]
    cache, o, pages, q, q64, rot, max_len = _attend_case(K, ctx, [61], B, n_q, H, G, lens, d, page, dtype, False)
    for b, sign in ((0, 1.0), (1, -1.0)):
        u = q[b, 0].float().mean(0)
        u = u / (u * u).sum()
        for t in range(lens[b]):
            cache.k[0, pages[b][t // page], 0, t % page] += (sign * 0.4 * t * d ** 0.5 * u).to(cache.dtype)
    o = dict(k=_f64(cache.k), v=_f64(cache.v))
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, lse=True)
    torch.cuda.synchronize()
    ref = O.attend(o, q64, pages, lens, d ** -0.5)
    _attend_close(_f64(out), _f64(lse), ref, dtype, d, lens, False)


def test_strided_queries_and_outputs(K, ctx):
    """Queries inside a projection's output, outputs with gaps: what lies between them is left alone."""
    B, n_q, H, G, d, page, lens = 3, 2, 2, 3, 128, 64, [500, 64, 3]
    cache, o, pages, _, _, rot, max_len = _attend_case(K, ctx, [71], B, n_q, H, G, lens, d, page, "bf16", True)
    rng = np.random.default_rng(3)
    big, b64 = _dev(rng.standard_normal((B, n_q, H * G + 4, d)), "bf16")
    q, q64 = big[:, :, :H * G], b64[:, :, :H * G]
    out = torch.full((n_q, B, H * G, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    got = ctx.paged_attend(cache, q, _ints(pages), _ints(lens), max_len, rope=rot, out=out.transpose(0, 1)[..., :d], scale=0.2)
    torch.cuda.synchronize()
    ref = O.attend(o, q64, pages, lens, 0.2, rot=_f64(rot))
    _attend_close(_f64(got), np.asarray(ref[1]), ref, "bf16", d, lens, True)
    assert bool((out[..., d:] == 7.0).all())


def test_a_decode_loop_in_a_graph(K, ctx):
    """Append with the rotation, then attend with it, captured once and replayed while sequences grow over page ends:
    every step against the oracle's, and a prompt appended at once gives the same cache as token by token."""
    B, H, G, d, page, steps, L = 3, 2, 4, 64, 16, 20, 2
    rng = np.random.default_rng(81)
    first = [0, 15, 30]
    total = [f + steps for f in first]
    n_pages = sum(-(-t // page) for t in total) + 1
    pages = _table(rng, n_pages, [-(-t // page) for t in total], 5)
    cache = ctx.paged_cache(L, n_pages, H, page, d)
    whole = ctx.paged_cache(L, n_pages, H, page, d)
    rot = ctx.rope_table(64, d, theta=1.0e4)
    new = torch.from_numpy(rng.standard_normal((2, L, B, H, max(total), d))).float().bfloat16().cuda()
    qs = torch.from_numpy(rng.standard_normal((steps, L, B, 1, H * G, d))).float().bfloat16().cuda()
    tab, start = _ints(pages), _ints(first)
    zero = _ints([0] * B)
    ctx.paged_append(whole, new[0], new[1], tab, zero, count=_ints(total), rope=rot)
    ctx.paged_append(cache, new[0], new[1], tab, zero, count=_ints(first), rope=rot)
    k1 = torch.empty((2, L, B, H, 1, d), dtype=torch.bfloat16, device="cuda")
    q1 = torch.empty((L, B, 1, H * G, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q1), torch.empty((L, B, 1, H * G), dtype=torch.float32, device="cuda")
    lens = start + 1
    ctx.paged_reserve(cache, B, 1, H * G, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for l in range(L):
            ctx.paged_append(cache, k1[0, l], k1[1, l], tab, start, layer=l, rope=rot)
            ctx.paged_attend(cache, q1[l], tab, lens, 64, layer=l, rope=rot, out=out[l], lse=lse[l])
        start += 1
        lens += 1
    for s in range(steps):
        at = torch.tensor([f + s for f in first], device="cuda")
        k1.copy_(torch.stack([new[:, :, b, :, int(at[b])] for b in range(B)], 2)[:, :, :, :, None])
        q1.copy_(qs[s])
        graph.replay()
        eager = ctx.paged_attend(cache, q1[1], tab, _ints([f + s + 1 for f in first]), 64, layer=1, rope=rot)
        torch.cuda.synchronize()
        assert torch.equal(eager, out[1])
        held = dict(k=_f64(cache.k), v=_f64(cache.v))
        now = [f + s + 1 for f in first]
        for l in range(L):
            ref = O.attend(held, _f64(qs[s, l]), pages, now, d ** -0.5, layer=l, rot=_f64(rot))
            _attend_close(_f64(out[l]), _f64(lse[l]), ref, "bf16", d, now, True, f"step {s} layer {l}")
    assert torch.equal(cache.k, whole.k) and torch.equal(cache.v, whole.v) and ctx.paged_dropped() == 0


def test_calls_on_another_stream(K, ctx):
    """What a call on a side stream allocates belongs to it, and its answers are the current stream's."""
    B, n_q, H, G, lens, d, page = 2, 1, 2, 4, [700, 33], 128, 64
    cache, o, pages, q, q64, rot, max_len = _attend_case(K, ctx, [91], B, n_q, H, G, lens, d, page, "bf16", True)
    tab, ln, zero = _ints(pages), _ints(lens), _ints([0, 0])
    want = ctx.paged_attend(cache, q, tab, ln, max_len, rope=rot, lse=True) + ctx.paged_read(cache, tab, zero, 33, rope=rot)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gone = {x.untyped_storage().data_ptr() for x in [torch.empty_like(w) for w in want for _ in range(4)]}
    turned = ctx.rope_table(rot.shape[0], d, theta=THETA, stream=side)
    got = ctx.paged_attend(cache, q, tab, ln, max_len, rope=turned, lse=True, stream=side) + \
        ctx.paged_read(cache, tab, zero, 33, rope=turned, stream=side)
    side.synchronize()
    assert not gone & {x.untyped_storage().data_ptr() for x in got}
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_a_pool_past_4_gib(K, ctx):
    """Pages whose offsets pass 32 bits, of the last layer."""
    page, d, H, L = 128, 128, 8, 2
    n_pages = 9000        # 2.36 GB a layer
    cache = ctx.paged_cache(L, n_pages, H, page, d)
    rng = np.random.default_rng(4)
    pages = [[n_pages - 1, 4500, n_pages - 2], [n_pages - 3, 1, 0]]
    start = [0, 0]
    n = 300
    k, v, k64, v64 = _rows(rng, 1, 2, H, n, d, "bf16", "tokens")
    rot = ctx.rope_table(n, d, theta=1.0e4)
    ctx.paged_append(cache, k, v, _ints(pages), _ints(start), layer=1, rope=rot)
    gk, gv = ctx.paged_read(cache, _ints(pages), _ints(start), n, layer=1, rope=None)
    torch.cuda.synchronize()
    assert np.array_equal(_f64(gv)[0], v64[0])
    size = np.stack([O.turn_size(k64[0, b], _f64(rot)) for b in range(2)])
    _turned_close(_f64(gk)[0], np.stack([O.turn(k64[0, b], _f64(rot)) for b in range(2)]), size, "bf16", "keys")
    assert int((cache.k[0] != 0).sum()) == 0 and int((cache.v[0] != 0).sum()) == 0
    q, q64 = _dev(rng.standard_normal((2, 1, H, d)), "bf16")
    out, lse = ctx.paged_attend(cache, q, _ints(pages), _ints([n, n]), n, layer=1, rope=rot, lse=True)
    small = dict(k=np.zeros((1, 6, H, page, d)), v=np.zeros((1, 6, H, page, d)))
    order = [[0, 1, 2], [3, 4, 5]]
    for b in range(2):
        for j in range(3):
            small["k"][0, order[b][j]] = _f64(cache.k[1, pages[b][j]])
            small["v"][0, order[b][j]] = _f64(cache.v[1, pages[b][j]])
    ref = O.attend(small, q64, order, [n, n], d ** -0.5, rot=_f64(rot))
    _attend_close(_f64(out), _f64(lse), ref, "bf16", d, [n, n], True)
