"""The ends of what the paged cache's calls take, on the CPU."""

import pytest

from cross_model_kv_amd import kvmap as K
from test_paged_boundary import _attend


@pytest.mark.parametrize("scale,status", [(2.35e38, K.OK), (2.4e38, K.ERR_INVALID_ARGUMENT), (3.4e38, K.ERR_INVALID_ARGUMENT),
                                          (1e-30, K.OK), (-1.0, K.ERR_INVALID_ARGUMENT)])
def test_scales(scale, status):
    """A scale whose product with log2 e is not an fp32 number would make every score an infinity or NaN."""
    assert _attend(scale=scale) == status
