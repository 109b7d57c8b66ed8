"""Tables of rotations that are a caller's own, or as long as they may be."""

import numpy as np
import pytest

from oracle import paged_oracle as O
from test_gpu_paged import _dev, _f64, _ints, _u

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    from cross_model_kv_amd import kvmap as K
    c = K.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stripping_scaled_rotations(ctx, dtype):
    """Keys that a table has turned and scaled come back times cos^2 + sin^2 by the same table, and as they were by one of cosines and
    sines over that.  Two roundings of an element by u, of products and sums in fp32 by 3 2^-24 each way, and of the tables' entries,
    4 2^-24, all of at most the pair's size (times the scale's square for the first)."""
    H, d, page, n = 2, 64, 16, 30
    g = np.random.default_rng(9)
    cache = ctx.paged_cache(1, 2, H, page, d, torch.bfloat16 if dtype == "bf16" else torch.float32)
    a, scale = g.uniform(0, 6.28, (n, d // 2)), g.uniform(0.5, 1.5, (n, 1))
    cs = np.stack([np.cos(a), np.sin(a)], -1) * scale[..., None]
    table, back = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (cs, cs / (scale * scale)[..., None]))
    k, k64 = _dev(g.standard_normal((1, H, n, d)), dtype)
    ctx.paged_append(cache, k, k, _ints([[1, 0]]), _ints([0]), rope=table)
    twice, _ = ctx.paged_read(cache, _ints([[1, 0]]), _ints([0]), n, rope=table)
    once, _ = ctx.paged_read(cache, _ints([[1, 0]]), _ints([0]), n, rope=back)
    torch.cuda.synchronize()
    size = np.sqrt(k64[0, ..., :d // 2] ** 2 + k64[0, ..., d // 2:] ** 2)
    size = 2 ** 0.5 * np.concatenate([size, size], -1)
    tol = (2 * _u(dtype) * (1 + _u(dtype)) + 10 * 2.0 ** -24) * size
    assert (abs(_f64(once)[0, 0] - k64[0]) <= tol).all()
    assert (abs(_f64(twice)[0, 0] - k64[0] * scale ** 2) <= tol * scale ** 2).all()


@pytest.mark.parametrize("n_pos,d", [(1 << 26, 128), ((1 << 26) - 3, 128), (1 << 26, 64)])
def test_the_longest_tables(ctx, n_pos, d):
    """Tables of 2^26 positions, more entries than a launch has work-items: every entry is written, and those at both ends and
    between are float64's cosines and sines to half a step of fp32, 2^-25, and the float64 angle's own two roundings of up to 2^-27
    each at 2^26."""
    table = ctx.rope_table(n_pos, d, theta=1.0e4, out=torch.full((n_pos, d // 2, 2), 7.0, device="cuda"))
    torch.cuda.synchronize()
    for part in table.split(1 << 22):
        assert bool((part.square().sum(-1) - 1).abs().le(1e-6).all())
    for at in (0, 12345678, 1 << 25, n_pos - 200):
        assert abs(_f64(table[at:at + 200]) - O.table(200, d, theta=1.0e4, pos0=at)).max() <= 2.0 ** -25 + 2 * 2.0 ** -27
    del table, part
    torch.cuda.empty_cache()
