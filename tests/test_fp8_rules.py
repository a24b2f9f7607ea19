"""Which kernel an FP8 product takes (host code alone, no GPU)."""
import os

import pytest

from w8a8_int8_quantized_absmax_amd import pdq

P = 1 << 20  # an address that is aligned and never read


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pdq.LIB_PATH):
        pytest.skip("libpdq.so not built")
    return pdq.lib()


@pytest.mark.parametrize("m,n,k", [(8, 8, 100), (8, 8, 8), (8, 8, 65552), ((1 << 21) + 1, 8, 64), (8, (1 << 21) + 1, 64), (1 << 21, 64, 65536),
                                   (64, 1 << 21, 65536), (1 << 20, (1 << 18) + 1, 64), (1 << 21, 1 << 21, 16), (-1, 8, 64), (8, 8, -16)])
def test_no_kernel_for_sizes_that_are_refused(L, m, n, k):
    # (bias is misaligned: nothing of what is accepted would be enqueued)
    assert L.pdq_gemm_fp8(P, P, m, k, P, P, 0, P + 2, n, P, 1, max(n, 1), None) == 2  # PDQ_ERR_SHAPE
    assert L.pdq_gemm_fp8_tile(m, n, k, 0) == -1 and L.pdq_gemm_fp8_tile(m, n, k, 1) == -1


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1 << 21, 1 << 17, 64), (1 << 17, 1 << 21, 128), (1 << 18, 64, 65536), (64, 1 << 18, 65536)])
def test_a_kernel_for_sizes_that_are_not(L, m, n, k):
    assert L.pdq_gemm_fp8(P, P, m, k, P, P, 0, P + 2, n, P, 1, n, None) == 4  # PDQ_ERR_ALIGN
    assert L.pdq_gemm_fp8_tile(m, n, k, 0) >= 0 and L.pdq_gemm_fp8_tile(m, n, k, 1) >= 0
