"""The 8-bit cache's oracle on the CPU: its rounding against torch's e4m3 conversion and against the
definition, its scales, and its attention against a direct softmax."""

import numpy as np
import pytest

from oracle import q8_oracle as Q

torch = pytest.importorskip("torch")


def test_code_values_match_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(Q.VALUE, t)


def test_rounding_matches_torch_and_is_nearest():
    rng = np.random.default_rng([2026, 801])
    x = np.concatenate([rng.standard_normal(20000) * s for s in (1e-3, 0.02, 1.0, 60.0)]).astype(np.float32)
    x = np.concatenate([x, ((Q._GRID[1:] + Q._GRID[:-1]) / 2).astype(np.float32), np.float32([0.0, -0.0, 448.0, -448.0])])
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(Q.e4m3_code(x.astype(np.float64)), want)
    err = np.abs(Q.VALUE[Q.e4m3_code(x)] - x)
    assert (err[:, None] <= np.abs(Q._GRID[None, :] - np.abs(x[:, None]))).all()


def test_what_is_not_finite_and_what_saturates():
    assert list(Q.e4m3_code([np.nan, np.inf, -np.inf, 500.0, -1e30])) == [0x7F, 0x7F, 0x7F, 0x7E, 0xFE]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (0.0, -110),
                                    (1e-40, -110), (3.3e38, 119)])
def test_scale_is_the_smallest_that_holds(amax, e):
    assert Q.scale_for(amax) == 2.0 ** e


def test_growth_rounds_what_was_held():
    c = Q.new_cache(1, 1, 1, 16, 64)
    one = np.full((1, 1, 1, 1, 64), 1.0)
    Q.write(c, one, one, [[0]], [0], [1])
    big = one * 1000
    Q.write(c, big, big, [[0]], [1], [1])
    s = Q.scale_for(1000.0)
    assert c["ks"][0, 0, 0] == s == c["vs"][0, 0, 0]
    np.testing.assert_array_equal(Q.tokens(c, "k", 0, 0, [0], 2)[0], Q.VALUE[Q.e4m3_code(1.0 / s)] * s)
    np.testing.assert_array_equal(Q.tokens(c, "v", 0, 0, [0], 2), Q.tokens(c, "k", 0, 0, [0], 2))


def test_pages_out_of_range_are_left_out():
    c = Q.new_cache(1, 2, 3, 16, 64)
    x = np.ones((1, 2, 3, 20, 64))
    # sequence 0: its second page is missing; sequence 1: a negative start
    assert Q.write(c, x, x, [[1, 2], [0, 0]], [0, -1], [20, 20]) == 2 * 3 * 2
    assert (c["ks"][0, 1] > 0).all() and (c["ks"][0, 0] == 0).all()


def test_attention_is_a_softmax_over_what_a_row_sees():
    rng = np.random.default_rng([2026, 802])
    c = Q.new_cache(2, 4, 2, 16, 64)
    x = rng.standard_normal((2, 2, 2, 2, 30, 64))
    pages, lens = [[2, 0], [3, 1]], [30, 2]
    Q.write(c, x[0], x[1], pages, [0, 0], lens)
    q = rng.standard_normal((2, 3, 4, 64))
    out, lse, _ = Q.attend(c, q, pages, lens, 1, 0.125)
    k, v = Q.read(c, pages, [0, 0], 30, lens, 1, 1)
    for b in range(2):
        for i in range(3):
            end = lens[b] - 3 + i + 1
            for h in range(4):
                if end <= 0:
                    assert (out[b, i, h] == 0).all() and lse[b, i, h] == -np.inf
                    continue
                y = torch.from_numpy(0.125 * (k[0, b, h // 2, :end] @ q[b, i, h]))
                np.testing.assert_allclose(out[b, i, h], torch.softmax(y, 0).numpy() @ v[0, b, h // 2, :end], rtol=1e-12)
                np.testing.assert_allclose(lse[b, i, h], torch.logsumexp(y, 0).item(), rtol=1e-12)
