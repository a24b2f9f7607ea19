"""Attention where one of its factors is near the end of its type's range, while the scores are ordinary."""
import numpy as np
import pytest

from kv_cases import Batch
from test_gpu_kv import run_attention

pytestmark = pytest.mark.gpu


def _batches(seed):
    yield Batch(seed, [200, 40, 1], None, 2, 128, 32, single=True)
    yield Batch(seed + 1, [150, 70], [140, 60], 2, 64, 16)
    yield Batch(seed + 2, [90], [70], 1, 256, 16)


def test_tiny_queries_over_large_scales():
    # bfloat16 goes down to 2^-126 and a page's scale up to 2^121; the products are ordinary scores
    for b in _batches(900):
        b.cache["k_scale"] *= np.float32(2.0 ** 125)  # 0.01 .. 0.05 before: 2^118 .. 2^121
        run_attention(b, 4, "bf16", spread=2.0 ** -123)
        run_attention(b, 4, "bf16", spread=2.0 ** -123, softcap=6.0)


def test_large_queries_over_tiny_scales():
    for b in _batches(910):
        b.cache["k_scale"] *= np.float32(2.0 ** -56)
        run_attention(b, 4, "bf16", spread=2.0 ** 56)
        run_attention(b, 4, "bf16", spread=2.0 ** 56, softcap=6.0)


def test_subnormal_binary16_queries():
    for b in _batches(920):
        run_attention(b, 4, "f16", spread=2.0 ** -18, scale=0.15 * 2.0 ** 17)


@pytest.mark.parametrize("rows", [1, 64])
def test_many_weights_far_below_the_largest(rows):
    # the first key has 2^20 times the weight of each of 6000 others, whose values are of the other sign: together they
    # move the result by 1.1%, each of them subnormal in binary16 beside the first
    n = 6000
    b = Batch(930 + rows, [n], [rows], 1, 64, 32)
    page = b.table[0, 0]
    b.cache["k_scale"][:] = b.cache["v_scale"][:] = 1 / 64
    b.cache["k"][:] = 0
    b.cache["v"][:] = 64
    b.cache["k"][page, 0, 0], b.cache["v"][page, 0, 0] = 64, -64
    rest = b.rows

    def ones(heads, dtype, scale):
        x = rest(heads, dtype, scale)
        return x * 0 + 1

    b.rows = ones
    run_attention(b, 2, "f16", scale=20 * np.log(2.0) / 64)


def test_tiny_caps():
    # far below any score, and still a cap: all of a row's keys weigh the same
    b = Batch(940, [70, 33], None, 2, 64, 16, single=True)
    b.cache["k"][b.table[0, 0], 0, 3:7] = 0  # products of zero among them
    run_attention(b, 4, "bf16", softcap=2.0 ** -100)
    b = Batch(941, [70], [60], 1, 128, 16)
    b.cache["k"][b.table[0, 0], 0, 3:7] = 0
    run_attention(b, 2, "f16", softcap=2.0 ** -100)
