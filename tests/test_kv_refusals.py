"""pdq_kv_attention's refusals of factors that its kernels could not form (nothing is enqueued, no pointer is followed)."""
import os

import pytest

from test_kv_abi import OK, UNSUP, att, batch
from w8a8_int8_quantized_absmax_amd import pdq


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pdq.LIB_PATH):
        pytest.skip("libpdq.so not built")
    return pdq.lib()


@pytest.mark.parametrize("scale,cap", [(0.1, 1e-40), (0.1, 1e-45), (-0.1, 1e-40), (0.0, 1e-45), (3e38, 0.0), (-3e38, 0.0),
                                       (1e20, 1e-19)])
def test_factors_that_are_not_finite(L, scale, cap):
    assert att(L, scale=scale, cap=cap, tokens=0, b=batch(batch=0, cu=None)) == UNSUP


@pytest.mark.parametrize("scale,cap", [(0.1, 2.0 ** -100), (2e38, 0.0), (0.0, 30.0), (1e10, 1e-19)])
def test_factors_that_are_finite(L, scale, cap):
    assert att(L, scale=scale, cap=cap, tokens=0, b=batch(batch=0, cu=None)) == OK
