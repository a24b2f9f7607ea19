"""Copies of the objects that hold tensors' addresses (MI355X): a copy's calls go by the copy's own."""
import copy
import io

import pytest
import torch

from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def saved(o):
    f = io.BytesIO()
    torch.save(o, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def randn(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).bfloat16().cuda()


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, saved])
def test_fp8(how):
    x, shared = randn(20, 256), how is copy.copy
    w, q, r = pdq.quantize_weight_fp8(randn(144, 256)), pdq.quantize_fp8(x), pdq.route_experts(randn(20, 4), 2)
    gate_up, down = pdq.quantize_weight_fp8(randn(4, 2, 128, 256)), pdq.quantize_weight_fp8(randn(4, 256, 128))
    y = [pdq.linear_fp8(x, w)["y"], pdq.gemm_fp8(q, w)["y"], pdq.experts_fp8(x, r, gate_up, down)["y"]]
    w2, q2, gate_up2, down2 = (how(o) for o in (w, q, gate_up, down))
    r2 = (copy.deepcopy if how is saved else how)(r)  # (torch.save refuses its two types in one buffer)
    for a, b in ((w.data, w2.data), (w.scale, w2.scale), (q.buffer, q2.buffer), (r.ids, r2.ids), (down.data, down2.data)):
        assert (a.data_ptr() == b.data_ptr()) == shared
    assert w2.at == w2.data.data_ptr() and w2.scale_at == w2.scale.data_ptr() and w2.shape == w.shape and gate_up2.shape == gate_up.shape
    if not shared:
        w.data.zero_(), q.buffer.zero_(), r.rows.fill_(-1), r.ids.fill_(-1), gate_up.data.zero_(), down.data.zero_()
    z = [pdq.linear_fp8(x, w2)["y"], pdq.gemm_fp8(q2, w2)["y"], pdq.experts_fp8(x, r2, gate_up2, down2)["y"]]
    assert all(torch.equal(a, b) for a, b in zip(y, z))


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, saved])
def test_cache(how):
    cache = pdq.KVCache.empty(4, 2, 64)
    batch = pdq.KVBatch(torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4), torch.full((1,), 3, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    x = randn(3, 2, 64)
    pdq.kv_append(x, x, cache, batch)
    y = pdq.kv_attention(x, cache, batch)["y"]
    cache2, batch2 = how(cache), how(batch)
    assert (cache2.k.data_ptr() == cache.k.data_ptr()) == (how is copy.copy)
    if how is not copy.copy:
        cache.k.zero_(), cache.v.zero_(), batch.seq_len.zero_()
    assert torch.equal(pdq.kv_attention(x, cache2, batch2)["y"], y)
