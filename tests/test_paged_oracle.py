"""Pins of the paged cache's oracle: hand-made cases, and attention against torch's own in float64."""

import numpy as np
import pytest

from oracle import paged_oracle as O


def test_a_quarter_turn():
    x = np.array([1.0, 2.0, 3.0, 4.0])
    cs = np.array([[0.0, 1.0], [1.0, 0.0]])          # pair 0 by 90 degrees, pair 1 not at all
    assert np.allclose(O.turn(x, cs), [-3.0, 2.0, 1.0, 4.0])
    assert np.allclose(O.turn(O.turn(x, cs), cs, -1.0), x)
    assert np.allclose(O.turn_size(x, cs), [3.0, 2.0, 1.0, 4.0])


def test_table_is_the_rotation():
    t = O.table(5, 8, theta=1e4, pos0=3)
    assert t.shape == (5, 4, 2)
    assert np.allclose(t[2, 1], [np.cos(5 * 1e4 ** -0.25), np.sin(5 * 1e4 ** -0.25)])
    assert np.allclose(O.table(2, 4, inv_freq=[0.5, 0.25])[1], [[np.cos(0.5), np.sin(0.5)], [np.cos(0.25), np.sin(0.25)]])


def test_scores_depend_on_distances_alone():
    rng = np.random.default_rng(0)
    q, k, t = rng.standard_normal(16), rng.standard_normal(16), O.table(40, 16, theta=100.0)
    assert np.isclose(O.turn(q, t[30]) @ O.turn(k, t[25]), O.turn(q, t[7]) @ O.turn(k, t[2]))


def _cache(rng, n_pages=6, H=2, page=4, d=8):
    return dict(k=rng.standard_normal((1, n_pages, H, page, d)), v=rng.standard_normal((1, n_pages, H, page, d)))


def test_append_then_read_gives_it_back():
    rng = np.random.default_rng(1)
    c, rot = _cache(rng), O.table(20, 8, theta=50.0)
    was = {x: c[x].copy() for x in "kv"}
    pages, start, count = [[3, 1, -1], [0, 9, 2]], [2, 3], [5, 3]
    k, v = rng.standard_normal((1, 2, 2, 6, 8)), rng.standard_normal((1, 2, 2, 6, 8))
    dropped, size = O.append(c, k, v, pages, start, count, rot=rot)
    assert dropped == 2                               # sequence 1's positions 4 and 5, in page 9
    assert np.array_equal(c["k"][:, [4, 5]], was["k"][:, [4, 5]]) and np.array_equal(c["v"][0, 3, :, :2], was["v"][0, 3, :, :2])
    rk, rv, _ = O.read(c, pages, start, 6, count, rot=rot)
    assert np.allclose(rk[0, 0, :, :5], k[0, 0, :, :5]) and np.array_equal(rv[0, 0, :, :5], v[0, 0, :, :5])
    assert not rk[0, 0, :, 5].any() and np.isnan(rk[0, 1, :, 1:3]).all() and not rv[0, 1, :, 3:].any()
    assert np.allclose(rk[0, 1, :, 0], k[0, 1, :, 0])


@pytest.mark.parametrize("rope", [False, True])
def test_attention_is_torchs(rope):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    c, rot = _cache(rng), O.table(24, 8, theta=50.0)
    pages, lens, n = [[5, 0, 2], [1, 4, 3]], [11, 2], 3
    q = rng.standard_normal((2, n, 4, 8))
    out, lse, size, prod = O.attend(c, q, pages, lens, 0.4, rot=rot if rope else None)
    for b in range(2):
        k = torch.from_numpy(c["k"][0][pages[b]].transpose(1, 0, 2, 3).reshape(2, 12, 8)[:, :lens[b]])
        v = torch.from_numpy(c["v"][0][pages[b]].transpose(1, 0, 2, 3).reshape(2, 12, 8)[:, :lens[b]])
        for i in range(n):
            pos = lens[b] - n + i
            if pos < 0:
                assert (lse[b, i] == -np.inf).all() and not out[b, i].any()
                continue
            x = torch.from_numpy(O.turn(q[b, i], rot[pos]) if rope else q[b, i])
            y = 0.4 * (x.view(2, 2, 8) @ k[:, :pos + 1].transpose(1, 2))
            assert np.allclose(torch.logsumexp(y, -1).reshape(4).numpy(), lse[b, i])
            assert np.allclose((torch.softmax(y, -1) @ v[:, :pos + 1]).reshape(4, 8).numpy(), out[b, i])
            assert (size[b, i] >= abs(out[b, i]) - 1e-12).all() and (prod[b, i] >= y.reshape(4, -1).amax(1).numpy() - 1e-12).all()
