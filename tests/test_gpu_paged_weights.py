"""Attention over the paged cache where a row's values nearly cancel: what is left shows how many bits its weights have.

Two tokens with scores y and 0, y from one product of a query's only element (a product of two bf16 numbers is exact in fp32),
and values c and -c' with c' the bf16 number nearest to c e^y.  Against float64, in units of 2^-24 of size = sum w |v|:
  an exponent y log2 e - m has the roundings of the scale's product with log2 e, of y's with it and of the difference, 3 |y|
  at most, and the exponential one of 2^-23, 2: the weights' errors;
  the products with all bits of a weight are exact but for their sums over two tokens and three parts, 3;
  the sum of the weights is rounded once, the quotient twice, 3;
and out is rounded once, u |ref|.
"""

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
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 20, 40])          # one tile of rows, two, and two blocks of two
@pytest.mark.parametrize("rope", [False, True])
def test_values_that_cancel(ctx, dtype, d, G, rope):
    from cross_model_kv_amd import kvmap as K
    B, H, page = 8, 16, 16
    rng = np.random.default_rng([d, G])
    bf16 = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
    y = bf16(rng.uniform(-2, 2, (B, H)))
    c = bf16(rng.uniform(1, 2, (B, H, d)))
    k, v = np.zeros((1, B, H, page, d)), np.zeros((1, B, H, page, d))
    k[0, :, :, 0, 0] = 1.0
    v[0, :, :, 0] = c
    v[0, :, :, 1] = -bf16(c * np.exp(y)[..., None])
    q = np.zeros((B, 1, H, G, d))
    q[:, 0, :, :, 0] = y[..., None]
    (kt, k64), (vt, v64), (qt, q64) = _dev(k, dtype), _dev(v, dtype), _dev(q.reshape(B, 1, H * G, d), dtype)
    pages, lens = [[b] for b in range(B)], [2] * B
    rot = torch.zeros((2, d // 2, 2), device="cuda") if rope else None      # turns by nothing
    if rope:
        rot[..., 0] = 1.0
    out = ctx.paged_attend(K.PagedCache(kt, vt), qt, _ints(pages), _ints(lens), 2, scale=1.0, rope=rot)
    torch.cuda.synchronize()
    ref, _, size, _ = O.attend(dict(k=k64, v=v64), q64, pages, lens, 1.0)
    tol = _u(dtype) * abs(ref) + (3 * 2 + 2 + 3 + 3) * 2.0 ** -24 * size
    err = abs(_f64(out) - ref)
    print(f"[paged weights] {dtype} d {d} G {G} rope {rope}: {(err / tol).max():.2f} of the tolerance", flush=True)
    assert (err <= tol).all(), f"{(err > tol).sum()} off, by up to {(err / tol).max():.1f} times the tolerance"
