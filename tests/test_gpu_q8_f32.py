"""fp32 calls of attention over the 8-bit cache keep 24 bits, on the GPU against the definition in 64 bits: the whole answer's error,
whose bound (q8_f32_cases.py) two bf16 parts of queries or weights do not meet (test_q8_parts.py)."""

import numpy as np
import pytest

from q8_f32_cases import CASES, WHOLE, case, whole
from test_gpu_q8 import _f64, _from_oracle, _ints
from test_gpu_q8_rows import reference

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


@pytest.mark.parametrize("lens,n_q,H,G,d,page", CASES)
def test_fp32_answers_keep_24_bits(ctx, K, lens, n_q, H, G, d, page):
    o, table, q = case(lens, n_q, H, G, d, page)
    out, lse = ctx.q8_attend(_from_oracle(K, o), torch.from_numpy(q.astype(np.float32)).cuda(), _ints(table), _ints(lens), max(lens), lse=True)
    ro, rl, _ = reference(o, q, table, lens, 0, d ** -0.5)
    seen = np.isfinite(rl)
    err = whole(_f64(out), ro)
    lerr = float(np.sqrt(np.mean((_f64(lse)[seen] - rl[seen]) ** 2)))
    print(f"[q8 f32] lens {lens} n_q {n_q} H {H} G {G} d {d} page {page}: {err:.2e} of its size, lse {lerr:.2e}", flush=True)
    assert err <= WHOLE
    assert lerr <= WHOLE * max(1.0, float(np.abs(rl[seen]).max()) / 8)   # (its own rounding is 2^-24 of it)
