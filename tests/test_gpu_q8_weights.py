"""Attention over the 8-bit cache where nearly all of a row's weight lies on tokens that add nothing to its answer, on the GPU
against the definition in 64 bits: language models put most of a row's weight on a first token whose values are near zero, and
the answer is made of the others, however far below they lie.

The bound on an output element, with w the weights and A = sum_t w_t |v_t| of its row and dim (a token with a value of zero adds
nothing to A, so A is of the answer's size here, whatever share of the weight such tokens have): the output's own rounding
u |ref|, and A times a weight's relative error and those of its score and of the sums (test_gpu_q8.py).  A weight in fewer bits than 8
would show here, where it counts as the largest do elsewhere: 2^-8; in fp32 calls it keeps 24.  There is no absolute term."""

import numpy as np
import pytest

from oracle import q8_oracle as Q
from test_gpu_q8 import _f64, _from_oracle, _ints, _rounded
from test_gpu_q8_rows import reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


def _bounds(out, lse, ref, T, d, dtype, where):
    ro, rl, f = ref
    u, w = (2.0 ** -8, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -24)
    delta = (d + 4) * 2.0 ** -24 * f["abss"] + 8 * 2.0 ** -24 * (1 + np.abs(rl))
    bound = u * np.abs(ro) + (w + 2 * delta[..., None] + T * 2.0 ** -24) * f["absv"]
    err, lerr = np.abs(_f64(out) - ro), np.abs(_f64(lse) - rl)
    worst, lworst = float((err / bound).max()), float((lerr / (delta + T * 2.0 ** -24 + 2.0 ** -24 * np.abs(rl))).max())
    norm = float(np.linalg.norm(_f64(out) - ro) / np.linalg.norm(ro))
    print(f"[q8 weights] {where}: out err/bound {worst:.3f}, of its size {norm:.2e}, lse err/bound {lworst:.3f}", flush=True)
    assert worst <= 1.0 and lworst <= 1.0, where


# Kernels by their rows of a KV head: decode's two, the prompt's of 128 rows and of 256.
SHAPES = [(1, 8, 128, 64, "bf16"), (3, 8, 128, 32, "bf16"), (2, 8, 64, 16, "bf16"), (30, 4, 128, 64, "bf16"), (40, 8, 128, 16, "bf16"),
          (50, 3, 64, 128, "bf16"), (1, 8, 128, 64, "f32"), (40, 2, 128, 64, "f32")]


def _case(rng, T, n_q, H, G, d, page, dtype, levels, zeros):
    """A sequence whose token t has scores `levels[t]` above a spread of about 1, values of mean 1, and zeros in `zeros[t]`'s
    dims; returns the oracle's cache, its table and the queries."""
    n_pages = -(-T // page)
    table = [[int(p) for p in rng.permutation(n_pages)]]
    x = rng.standard_normal((2, 1, 1, H, T, d))
    x[1] = 1 + 0.5 * x[1]
    x[0, ..., 0] = levels / (8 * d ** -0.5)
    for dims, at in zeros:
        x[1][..., at[:, None], dims] = 0.0
    o = Q.new_cache(1, n_pages, H, page, d)
    Q.write(o, x[0], x[1], table, [0], [T])
    q = rng.standard_normal((1, n_q, H * G, d))
    q[..., 0] = 8
    return o, table, _rounded(q, dtype)


def _run(ctx, o, table, q, T, d, dtype, where):
    from cross_model_kv_amd import kvmap as K
    out, lse = ctx.q8_attend(_from_oracle(K, o), q, _ints(table), _ints([T]), T, lse=True)
    _bounds(out, lse, reference(o, _f64(q), table, [T], 0, d ** -0.5), T, d, dtype, where)


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
@pytest.mark.parametrize("nats", [14, 18, 22, 26])
def test_a_first_token_with_nearly_all_weight(ctx, nats, n_q, G, d, page, dtype):
    T = 4100
    rng = np.random.default_rng([2026, 871, nats, n_q, G, d, page])
    levels = np.zeros(T)
    levels[0] = nats
    o, table, q = _case(rng, T, n_q, 2, G, d, page, dtype, levels, [(slice(None), np.array([0]))])
    _run(ctx, o, table, q, T, d, dtype, f"first token {nats} nats up, n_q {n_q} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
def test_tokens_with_nearly_all_weight_anywhere(ctx, n_q, G, d, page, dtype):
    """One in every 40 tokens lies up to 20 nats above the others, so that each tile of tokens has its own, and long stretches lie as
    much lower than the rest."""
    T = 3000
    rng = np.random.default_rng([2026, 872, n_q, G, d, page])
    high = np.unique(rng.integers(0, T - n_q, T // 40))
    levels = np.zeros(T)
    levels[1000:1700] = -9
    levels[high] += rng.uniform(12, 20, len(high))
    o, table, q = _case(rng, T, n_q, 2, G, d, page, dtype, levels, [(slice(None), high)])
    _run(ctx, o, table, q, T, d, dtype, f"one in 40 up to 20 nats up, n_q {n_q} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
def test_stretches_at_levels_of_their_own(ctx, n_q, G, d, page, dtype):
    """Stretches of tokens up to 30 nats apart, up and down again, each with values in dims of its own: what a dim's answer is made of
    may lie at any level."""
    T, parts = 2400, 8
    rng = np.random.default_rng([2026, 873, n_q, G, d, page])
    part = np.arange(T) * parts // T
    levels = np.array([0, 20, -8, 12, 22, -3, 8, -6])[part]
    zeros = [(np.flatnonzero(np.arange(d) % parts != i), np.flatnonzero(part == i)) for i in range(parts)]
    o, table, q = _case(rng, T, n_q, 1, G, d, page, dtype, levels, zeros)
    _run(ctx, o, table, q, T, d, dtype, f"stretches, n_q {n_q} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
@pytest.mark.parametrize("nats", [9, 11, 12.1, 12.7, 13.3, 17, 40])
def test_equal_scores_far_below_the_first_ones(ctx, nats, n_q, G, d, page, dtype):
    """After 96 tokens with values of zero, all scores are equal: a rounding of their weights would be the same for all of them."""
    T = 1000
    rng = np.random.default_rng([2026, 875, int(10 * nats), n_q, G, d, page])
    levels = np.full(T, -float(nats))
    levels[:96] = 0
    o, table, q = _case(rng, T, n_q, 2, G, d, page, dtype, levels, [(slice(None), np.arange(96))])
    q[..., 1:] = 0
    _run(ctx, o, table, q, T, d, dtype, f"equal scores {nats} nats below, n_q {n_q} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
@pytest.mark.parametrize("before,nats", [(16, 9), (16, 11.5), (16, 12.6), (16, 20), (32, 12.6), (40, 10), (1, 14), (1, 30)])
def test_a_rows_own_tokens_far_below_the_first_ones(ctx, before, nats, n_q, G, d, page, dtype):
    """Only the first tokens are seen by all rows, and they have values of zero: a row's answer is made of the queries' own tokens up to
    it, one for the first row, a part of 16 for most."""
    T = before + n_q
    rng = np.random.default_rng([2026, 876, before, int(10 * nats), n_q, G, d, page])
    levels = np.full(T, -float(nats))
    levels[:before] = 0
    o, table, q = _case(rng, T, n_q, 2, G, d, page, dtype, levels, [(slice(None), np.arange(before))])
    _run(ctx, o, table, q, T, d, dtype, f"own tokens {nats} nats below {before}, n_q {n_q} G {G} d {d} page {page} {dtype}")


@pytest.mark.parametrize("n_q,G,d,page,dtype", SHAPES)
def test_one_page_of_much_larger_values(ctx, n_q, G, d, page, dtype):
    """A page whose values are 2^24 times the others' in one dim and zeros in the rest: its scale is as much larger, which must not cost
    the other pages anything."""
    T = 1500
    rng = np.random.default_rng([2026, 874, n_q, G, d, page])
    o, table, q = _case(rng, T, n_q, 2, G, d, page, dtype, np.zeros(T), [])
    at = slice(5 * page, 6 * page)
    x = np.zeros((2, 1, 1, 2, page, d))
    x[0] = rng.standard_normal(x[0].shape)
    x[1, ..., 3] = 2.0 ** 24 * (1 + 0.2 * rng.standard_normal(x[1, ..., 3].shape))
    Q.write(o, x[0], x[1], table, [at.start], [page])
    _run(ctx, o, table, q, T, d, dtype, f"one page of large values, n_q {n_q} G {G} d {d} page {page} {dtype}")
