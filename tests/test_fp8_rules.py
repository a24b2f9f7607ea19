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


# (rows of the tile, 0: few rows; measured times of few rows / 128 x 128 / 128 x 256 / 256 x 256 or 192 x 256, microseconds)
@pytest.mark.parametrize("m,n,k,scales,tile", [
    (600, 2048, 11008, 0, 0), (768, 2048, 14336, 0, 0),        # 40.9 / 49.5; 53.5 / 72.0
    (8192, 4096, 128, 1, 128),                                 # 52.7 / 24.9 / 27.5
    (400, 3008, 4096, 0, 128), (400, 3008, 4096, 1, 128),      # 23.0 / 17.8; 24.7 / 20.6
    (601, 1003, 1360, 1, 0), (601, 1003, 1360, 0, 0),          # 7.7 / 15.1; 8.4 / 12.9
    (512, 4096, 4096, 1, 128), (256, 4096, 4096, 1, 0),        # 23.8 / 21.5; 14.6 / 19.6
    (100, 4096, 4096, 0, 0), (4096, 11008, 4096, 0, 256), (8192, 4096, 14336, 1, 192), (1024, 4096, 14336, 0, 128)])
def test_the_faster_kernel(L, m, n, k, scales, tile):
    assert L.pdq_gemm_fp8_tile(m, n, k, scales) == tile


@pytest.mark.parametrize("scales", [0, 1])
def test_tiles_for_many_rows_of_little_depth(L, scales):
    # 65536 x 4096, one group: 396 / 179 / 187 / 186, with binary32 scales 426 / 187 / 200.  The largest products: the kernel for few rows
    # would take more threads than a launch has
    for m, n in ((65536, 4096), (1 << 21, 1 << 17), (1 << 17, 1 << 21), (1 << 19, 1 << 19), ((1 << 20) + 5, 200003)):
        for k in (16, 128, 1024):
            assert L.pdq_gemm_fp8_tile(m, n, k, scales) > 0
