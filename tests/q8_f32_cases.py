"""fp32 cases of attention over the 8-bit cache, and the bound on a whole answer, shared by the test of the kernels and the test of the
bound."""

import numpy as np

from test_gpu_q8 import _held

# Queries and weights in three bf16 parts are off by 2^-24 of themselves, as fp32 is.  Then there are the roundings of a score (some
# 12 sums of its parts, and the exponent's argument, of size |y| <= 8 or so) and of the sums over tokens, 2^-24 each and
# independent: 10 to 16 of them in the mean square.  Two parts are off by up to 2^-16, 2^-18 in the mean square: 64 times 2^-24.
WHOLE = 16 * 2.0 ** -24

CASES = [
    # lens, n_q, H, G, d, page
    ([300], 1, 2, 8, 128, 64),
    ([1000, 3], 1, 2, 3, 64, 32),
    ([255, 256, 257, 511], 1, 1, 16, 128, 128),
    ([700, 80], 3, 2, 8, 64, 16),
    ([300, 7, 0], 9, 2, 3, 128, 32),
    ([257], 129, 1, 2, 64, 16),
    ([70, 300], 70, 2, 3, 128, 32),
    ([300], 300, 1, 3, 128, 16),
    ([6000, 2000], 1, 4, 4, 128, 64),
    ([4000, 1500], 40, 2, 2, 64, 64),
]


def case(lens, n_q, H, G, d, page):
    """The oracle's cache, its table and float64 queries that fp32 holds."""
    rng = np.random.default_rng([2026, 901, len(lens), max(lens), n_q, H, G, d, page])
    o, table = _held(rng, lens, H, page, d)
    return o, table, rng.standard_normal((len(lens), n_q, H * G, d)).astype(np.float32).astype(np.float64)


def whole(got, ref):
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
