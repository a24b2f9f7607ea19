"""Objects that hold checked addresses and sizes refuse what would leave those behind (no GPU)."""
import pytest

from w8a8_int8_quantized_absmax_amd import pdq


def slots(cls):
    return [s for c in cls.__mro__ for s in getattr(c, "__slots__", ())]


@pytest.mark.parametrize("cls", [pdq.WeightFP8, pdq.CodesFP8, pdq.Routing])
def test_no_attribute_can_be_set(cls):
    o = cls.__new__(cls)
    names = slots(cls)
    assert len(names) >= 6
    for name in names + ["something"]:
        with pytest.raises(AttributeError, match="cannot be set"):
            setattr(o, name, 1)
    o._put(**{names[0]: 7})  # as their own code does
    assert getattr(o, names[0]) == 7
    with pytest.raises(AttributeError, match="cannot be deleted"):
        delattr(o, names[0])


@pytest.mark.parametrize("cls", [pdq.KVCache, pdq.KVBatch])
def test_no_attribute_of_a_cache_can_be_set(cls):
    test_no_attribute_can_be_set(cls)


@pytest.mark.gpu
def test_of_the_objects_that_calls_make():
    import torch

    x = torch.ones((20, 256), dtype=torch.bfloat16, device="cuda")
    w, q = pdq.quantize_weight_fp8(x), pdq.quantize_fp8(x)
    r = pdq.route_experts(x[:, :8], 2)
    y = pdq.linear_fp8(x, w)["y"]
    for o, names in ((w, ("data", "scale", "n", "k", "lead", "at")), (q, ("buffer", "rows", "k")),
                     (r, ("tokens", "experts", "k", "ids", "weights"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(o, name, getattr(o, name))
    w.scale.view(torch.uint8).add_(1)  # in place: twice the weight
    assert torch.equal(pdq.linear_fp8(x, w)["y"], 2 * y) and torch.equal(pdq.gemm_fp8(q, w)["y"], 2 * y)
    assert type(r) is pdq.Routing and r.ids.shape == (20, 2) and type(q) is pdq.CodesFP8 and q.shape == (20, 256)


@pytest.mark.gpu
def test_of_a_cache_and_its_batch():
    import torch

    cache = pdq.KVCache.empty(4, 2, 64)
    batch = pdq.KVBatch(torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"))
    for o, names in ((cache, ("k", "v", "k_scale", "pages", "dim")), (batch, ("page_table", "seq_len", "cu_q", "batch"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(o, name, getattr(o, name))
    x = torch.randn((1, 2, 64), device="cuda").bfloat16()
    pdq.kv_append(x, x, cache, batch)
    assert torch.isfinite(pdq.kv_attention(x, cache, batch)["y"]).all()
