"""The row-at-once reference of the GPU tests against the oracle, on the CPU."""

import numpy as np
import pytest

from oracle import q8_oracle as Q

pytest.importorskip("torch")


def test_reference_is_the_oracle():
    from test_gpu_q8 import _held
    from test_gpu_q8_rows import reference
    rng = np.random.default_rng([2026, 851])
    lens, n, H, G, d = [21, 3, 0, 16], 5, 2, 3, 64
    o, table = _held(rng, lens, H, 16, d)
    q = rng.standard_normal((4, n, H * G, d))
    a, b = Q.attend(o, q, table, lens, 0, 0.1), reference(o, q, table, lens, 0, 0.1)
    for x, y in [(a[0], b[0]), (a[1], b[1])] + [(a[2][k], b[2][k]) for k in a[2]]:
        np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-300)
