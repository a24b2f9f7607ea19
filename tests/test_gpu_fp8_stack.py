"""Single matrices of a stack of FP8 weights, as a C caller takes them out of it."""
import os

import pytest
import torch

from w8a8_int8_quantized_absmax_amd import pdq

P = 1 << 20  # an address that is aligned and never read


def test_scales_of_a_matrix_within_a_stack():
    if not os.path.exists(pdq.LIB_PATH):
        pytest.skip("libpdq.so not built")
    L = pdq.lib()

    def f(n, k, i, scale_t):  # (no rows: nothing is enqueued)
        at = i * ((n + 127) // 128) * L.pdq_fp8_scale_pitch(k) * (4 if scale_t else 1)
        return at % 16, L.pdq_gemm_fp8(P, P, 0, k, P + i * L.pdq_fp8_bytes(n, k), P + at, scale_t, None, n, P, 1, n, None)

    assert f(256, 256, 1, 0) == (8, 4) and f(256, 256, 2, 0) == (0, 0)     # PDQ_ERR_ALIGN, PDQ_OK
    assert f(512, 256, 1, 0) == (0, 0) and f(128, 2048, 3, 0) == (0, 0)
    for i in range(4):
        assert f(16, 16, i, 1) == (0, 0) and f(300, 400, i, 1) == (0, 0)   # binary32 ones always


@pytest.mark.gpu
@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("m", [3, 40, 700])
def test_products_by_each_matrix_of_a_stack(m, scales):
    count, n, k = 3, 512, 400
    g = torch.Generator().manual_seed(m)
    codes = torch.randn((count, n, k), generator=g).mul(40).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    s = torch.exp2(torch.randint(-12, -8, (count, 4, 4), generator=g).float()).cuda()
    s = s if scales == "f32" else s.to(torch.float8_e8m0fnu)
    stack = pdq.pack_weight_fp8(codes, s)
    x = pdq.quantize_fp8(torch.randn((m, k), generator=g).bfloat16().cuda())
    at, pitch = x.buffer.data_ptr(), stack.scale.shape[-1] * stack.scale.element_size()
    for i in range(count):
        y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        pdq._kv_call("pdq_gemm_fp8", 0, at, at + x.size, m, k, stack.data.data_ptr() + i * pdq.fp8_bytes(n, k),
                     stack.scale.data_ptr() + i * 4 * pitch, stack.scale_type, None, n, y.data_ptr(), 1, n)
        one = pdq.pack_weight_fp8(codes[i].contiguous(), s.view(torch.uint8)[i].contiguous().view(s.dtype) if scales == "pow2" else s[i].contiguous())
        assert torch.equal(y, pdq.gemm_fp8(x, one)["y"])
