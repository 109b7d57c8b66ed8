"""Attention over the 8-bit cache for many rows (prompts, drafts), and for many sequences at once, on the GPU against
the definition in 64 bits.  The error bounds are those derived in test_gpu_q8.py."""

import numpy as np
import pytest

from oracle import q8_oracle as Q
from test_gpu_q8 import _check, _f64, _from_oracle, _held, _ints, _rounded, _rows

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


def reference(c, q, pages, lens, layer, scale):
    """What q8_oracle.attend gives, all rows of a sequence and KV head at once."""
    B, n, Hq, d = q.shape
    H, P = c["k"].shape[2], c["k"].shape[3]
    G = Hq // H
    out, absv = np.zeros((B, n, Hq, d)), np.zeros((B, n, Hq, d))
    lse, abss, wv = np.full((B, n, Hq), -np.inf), np.zeros((B, n, Hq)), np.zeros((B, n, Hq))
    for b in range(B):
        T = int(lens[b])
        if not T:
            continue
        vs = np.array([c["vs"][layer, p] if 0 <= p < c["vs"].shape[1] else np.full(H, np.nan)
                       for p in pages[b][:-(-T // P)]]).repeat(P, axis=0)[:T]
        ahead = np.arange(T) > (T - n + np.arange(n))[:, None]                    # [n][T]
        for h in range(H):
            k, v = Q.tokens(c, "k", layer, h, pages[b], T), Q.tokens(c, "v", layer, h, pages[b], T)
            rows = q[b, :, h * G:(h + 1) * G].transpose(1, 0, 2)                   # [G][n][d]
            y = np.where(ahead, -np.inf, scale * (rows @ k.T))
            m = y.max(-1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            p = np.exp(y - m)
            s = p.sum(-1, keepdims=True)
            w = p / np.where(s > 0, s, 1.0)
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            with np.errstate(divide="ignore"):
                lse[at] = (m + np.log(s))[..., 0].T
            out[at], absv[at] = (w @ v).transpose(1, 0, 2), (w @ np.abs(v)).transpose(1, 0, 2)
            abss[at] = np.where(ahead, 0.0, scale * (np.abs(rows) @ np.abs(k).T)).max(-1).T
            wv[at] = (w * vs[:, h]).max(-1).T
    return out, lse, dict(absv=absv, abss=abss, wv=wv)


ROWS = [
    # lens, n_q, H, G, d, page, dtype
    ([40], 33, 1, 1, 128, 64, "bf16"),
    ([33], 33, 1, 1, 64, 16, "f32"),
    ([2, 0, 1], 40, 1, 1, 128, 16, "bf16"),
    ([129, 5, 0], 129, 1, 1, 128, 16, "bf16"),
    ([300], 128, 2, 1, 128, 64, "bf16"),
    ([300], 129, 2, 1, 128, 64, "bf16"),
    ([600, 0, 257, 1], 257, 1, 1, 128, 32, "bf16"),
    ([700, 64, 65], 65, 2, 8, 128, 64, "bf16"),
    ([700, 63, 127], 65, 2, 8, 64, 128, "bf16"),
    ([5000, 37], 16, 2, 3, 128, 128, "bf16"),
    ([5000, 37], 16, 2, 3, 64, 64, "bf16"),
    ([9001], 7, 1, 5, 128, 64, "bf16"),
    ([2000, 100], 12, 2, 4, 128, 32, "f32"),
    ([700, 9], 90, 2, 2, 64, 128, "f32"),
    ([300], 300, 3, 3, 128, 16, "f32"),
    ([2500, 300, 1], 300, 2, 4, 128, 64, "bf16"),
    ([2048], 512, 1, 2, 128, 128, "bf16"),
    ([64], 64, 16, 3, 64, 32, "bf16"),
]


@pytest.mark.parametrize("lens,n_q,H,G,d,page,dtype", ROWS)
def test_rows_match_the_definition(ctx, K, lens, n_q, H, G, d, page, dtype):
    rng = np.random.default_rng([2026, 841, len(lens), max(lens), n_q, H, G, d, page])
    o, table = _held(rng, lens, H, page, d, L=2, layer=1, sharp=2.0)
    c = _from_oracle(K, o)
    q = _rounded(1.5 * rng.standard_normal((len(lens), n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), max(lens) + page, layer=1, lse=True)
    ref = reference(o, _f64(q), table, lens, 1, d ** -0.5)
    _check(out, lse, ref, max(lens), d, dtype, f"lens {lens} n_q {n_q} H {H} G {G} d {d} page {page} {dtype}")
    again, lse2 = ctx.q8_attend(c, q, _ints(table), _ints(lens), max(lens) + page, layer=1, lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,n_q,H,G,d,page,top,dtype", [
    (70, 40, 4, 1, 128, 16, 200, "bf16"),      # more items than workgroups, more sequences than a wave has lanes
    (130, 1, 2, 4, 128, 32, 900, "bf16"),
    (200, 3, 1, 5, 64, 16, 300, "bf16"),
    (67, 1, 3, 2, 64, 64, 2000, "f32"),
    (90, 20, 8, 2, 64, 16, 150, "bf16"),
])
def test_many_sequences(ctx, K, B, n_q, H, G, d, page, top, dtype):
    """Unequal lengths, zeros and ones among them, and the longest one alone far above the others."""
    rng = np.random.default_rng([2026, 842, B, n_q, H])
    lens = [int(x) for x in rng.integers(0, top // 4, B)]
    lens[1], lens[2], lens[B // 2], lens[-1] = 0, 1, top, 0
    o, table = _held(rng, lens, H, page, d)
    c = _from_oracle(K, o)
    q = _rounded(1.5 * rng.standard_normal((B, n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints(lens), top + 1, lse=True)
    _check(out, lse, reference(o, _f64(q), table, lens, 0, d ** -0.5), top, d, dtype, f"B {B} n_q {n_q} H {H} G {G}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,T", [(1, 4000), (20, 3000), (100, 1500)])
def test_nan_where_pieces_meet(ctx, K, dtype, n_q, T):
    """NaN codes among the newest tokens and far before them, in a sequence that is worked on in pieces: the rows that see
    one become NaN, in the dims that hold it; a page out of range makes all of them NaN."""
    rng = np.random.default_rng([2026, 843, n_q, T])
    H, G, d, page = 2, 3, 128, 64
    o, table = _held(rng, [T], H, page, d)
    q = _rounded(rng.standard_normal((1, n_q, H * G, d)), dtype)
    clean = reference(o, _f64(q), table, [T], 0, d ** -0.5)
    early, late = T // 3, T - 1
    o["v"][0, table[0][early // page], 0, 7, early % page] = 0x7F          # head 0: an old value that all rows see,
    o["v"][0, table[0][late // page], 0, [0, 33, 127], late % page] = 0xFF  # and the newest one's
    c = _from_oracle(K, o)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints([T]), T, lse=True)
    nan = np.zeros((1, n_q, H * G, d), bool)
    nan[0, :, :G, 7] = True
    nan[0, -1, :G, [0, 33, 127]] = True
    np.testing.assert_array_equal(np.isnan(_f64(out)), nan)
    at = torch.from_numpy(nan).cuda()
    out[at] = torch.from_numpy(clean[0]).to(out)[at]
    _check(out, lse, clean, T, d, dtype, f"NaN n_q {n_q} T {T} {dtype}")
    gone = [list(table[0])]
    gone[0][2] = -1
    out, lse = ctx.q8_attend(c, q, _ints(gone), _ints([T]), T, lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 30])
def test_values_with_the_smallest_scales(ctx, K, dtype, n_q):
    """Values of 1e-31: their scales lie below those that the weights are held with."""
    rng = np.random.default_rng([2026, 844, n_q])
    H, G, d, page, T = 2, 2, 128, 32, 200
    o, table = _held(rng, [T], H, page, d)
    o["vs"][:] = 2.0 ** rng.integers(-110, -95, o["vs"].shape)
    c = _from_oracle(K, o)
    q = _rounded(rng.standard_normal((1, n_q, H * G, d)), dtype)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints([T]), T, lse=True)
    ref = reference(o, _f64(q), table, [T], 0, d ** -0.5)
    _check(out, lse, ref, T, d, dtype, f"smallest scales n_q {n_q} {dtype}")
    assert (np.abs(_f64(out)) > 0).any()


def test_lengths_out_of_range_beside_prompts(ctx, K):
    rng = np.random.default_rng([2026, 845])
    lens, H, G, d, page, n_q = [300, 120, 0, 77], 2, 4, 128, 64, 50
    o, table = _held(rng, lens, H, page, d)
    c = _from_oracle(K, o)
    q = _rounded(rng.standard_normal((4, n_q, H * G, d)), "bf16")
    want = reference(o, _f64(q), table, lens, 0, d ** -0.5)
    out, lse = ctx.q8_attend(c, q, _ints(table), _ints([300, -3, 0, 301]), 300, lse=True)
    for b in (1, 3):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
    part = (want[0][[0, 2]], want[1][[0, 2]], {k: x[[0, 2]] for k, x in want[2].items()})
    _check(out[[0, 2]], lse[[0, 2]], part, 300, d, "bf16", "beside sequences out of range")


def test_prompt_in_a_graph(ctx, K):
    """Write and attend of 24 rows' queries captured once and replayed over growing sequences, eager calls in between."""
    rng = np.random.default_rng([2026, 846])
    H, G, d, page, n_q, steps = 2, 4, 128, 64, 12, 5
    lens, max_len = [0, 700], 1024
    table = [list(range(16)), list(range(16, 32))]
    new = [_rows(rng, 1, 2, H, n_q, d, "bf16", "tokens", spread=0.3)[:2] for _ in range(steps)]
    qs = _rounded(rng.standard_normal((steps, 2, n_q, H * G, d)), "bf16")
    eager, replayed = ctx.q8_cache(1, 32, H, page, d), ctx.q8_cache(1, 32, H, page, d)
    k0, v0 = _rows(rng, 1, 2, H, 700, d, "bf16", "heads", spread=0.3)[:2]
    pages = _ints(table)
    for c in (eager, replayed):
        ctx.q8_write(c, k0, v0, pages, _ints([0, 0]), count=_ints(lens))
    ctx.q8_reserve(eager, 2, n_q, H * G, max_len)
    k, v, q = new[0][0].clone(), new[0][1].clone(), qs[0].clone()
    start, held = _ints(lens), _ints(lens)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.q8_write(replayed, k, v, pages, start)
        ctx.q8_attend(replayed, q, pages, held, max_len, out=out)
    for s in range(steps):
        now = [t + s * n_q for t in lens]
        ctx.q8_write(eager, new[s][0], new[s][1], pages, _ints(now))
        want = ctx.q8_attend(eager, qs[s], pages, _ints([t + n_q for t in now]), max_len)
        k.copy_(new[s][0])
        v.copy_(new[s][1])
        q.copy_(qs[s])
        start.copy_(_ints(now))
        held.copy_(_ints([t + n_q for t in now]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), s
