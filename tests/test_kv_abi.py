"""The key/value cache's entry points on the host: refusals (nothing is enqueued, no pointer is followed) and the
oracle's own properties."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
from w8a8_int8_quantized_absmax_amd import pdq

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
P = 0x10000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pdq.LIB_PATH):
        pytest.skip("libpdq.so not built")
    return pdq.lib()


def cache(k=P, v=P, ks=P, vs=P, pages=8, heads=2, page=16, dim=64):
    return ctypes.byref(pdq._KVCacheC(k, v, ks, vs, pages, heads, page, dim))


def batch(table=P, ldt=4, seq_len=P, cu=P, batch=3, max_pages=4):
    return ctypes.byref(pdq._KVBatchC(table, ldt, seq_len, cu, batch, max_pages))


def app(L, k=P, v=P, q=P, dt=1, tokens=5, hq=4, ldk=128, ldv=128, ldq=256, cos=P, sin=P, positions=64, rot=64,
        inter=0, c=None, b=None, q_out=P, ldqo=256):
    return L.pdq_kv_append(k, v, q, dt, tokens, hq, ldk, ldv, ldq, cos, sin, positions, rot, inter,
                           c or cache(), b or batch(), q_out, ldqo, None)


def att(L, q=P, dt=1, tokens=5, hq=4, ldq=256, c=None, b=None, scale=0.1, cap=0.0, window=0, slopes=None,
        prefix=None, y=P, ldy=256, lse=None, ws=P, ws_bytes=1 << 40):
    return L.pdq_kv_attention(q, dt, tokens, hq, ldq, c or cache(), b or batch(), scale, cap, window, slopes, prefix,
                              y, ldy, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [app, att])
def test_cache_and_batch_refusals(L, call):
    for bad in (dict(pages=-1), dict(pages=1 << 31), dict(heads=0), dict(heads=257), dict(page=8), dict(page=48),
                dict(page=512), dict(dim=96), dict(dim=0), dict(dim=512)):
        assert call(L, c=cache(**bad)) == SHAPE, bad
    for bad in (dict(batch=-1), dict(batch=65537), dict(max_pages=-1), dict(ldt=3), dict(max_pages=1 << 27, ldt=1 << 27),
                dict(cu=None)):
        assert call(L, b=batch(**bad)) == SHAPE, bad
    assert call(L, tokens=-1) == SHAPE
    assert call(L, tokens=(1 << 21) + 1) == SHAPE
    for bad in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None)):
        assert call(L, c=cache(**bad)) == NULL, bad
    for bad in (dict(table=None), dict(seq_len=None)):
        assert call(L, b=batch(**bad)) == NULL, bad
    for bad in (dict(k=P + 8), dict(v=P + 4), dict(ks=P + 2), dict(vs=P + 1)):
        assert call(L, c=cache(**bad)) == ALIGN, bad
    for bad in (dict(table=P + 2), dict(seq_len=P + 1), dict(cu=P + 2)):
        assert call(L, b=batch(**bad)) == ALIGN, bad
    for dt in (0, 3, -1):
        assert call(L, dt=dt) == DTYPE
    assert call(L, tokens=0, b=batch(batch=0, cu=None)) == OK  # nothing to do, nothing launched
    assert call(L, tokens=0) == OK


def test_null_structs(L):
    assert L.pdq_kv_append(P, P, None, 1, 5, 0, 128, 128, 0, None, None, 0, 0, 0, None, batch(), None, 0, None) == NULL
    assert L.pdq_kv_attention(P, 1, 5, 4, 256, cache(), None, 0.1, 0.0, 0, None, None, P, 256, None, P, 1 << 40,
                              None) == NULL


def test_append_refusals(L):
    assert app(L, k=None) == NULL
    assert app(L, v=None) == NULL
    assert app(L, q_out=None) == NULL
    assert app(L, cos=None) == NULL
    assert app(L, sin=None) == NULL
    assert app(L, cos=None, sin=None) == NULL  # queries are there to be rotated
    assert app(L, ldk=120) == SHAPE
    assert app(L, ldv=120) == SHAPE
    assert app(L, ldq=248) == SHAPE
    assert app(L, ldqo=248) == SHAPE
    assert app(L, hq=0) == SHAPE
    assert app(L, rot=8) == SHAPE
    assert app(L, rot=40) == SHAPE
    assert app(L, rot=80) == SHAPE
    assert app(L, positions=0) == SHAPE
    assert app(L, k=P + 8) == ALIGN
    assert app(L, v=P + 2) == ALIGN
    assert app(L, q=P + 4) == ALIGN
    assert app(L, q_out=P + 8) == ALIGN
    assert app(L, cos=P + 4) == ALIGN
    assert app(L, sin=P + 8) == ALIGN
    assert app(L, ldk=132) == ALIGN
    assert app(L, ldq=260) == ALIGN


def test_attention_refusals(L):
    assert att(L, q=None) == NULL
    assert att(L, y=None) == NULL
    assert att(L, hq=3) == SHAPE
    assert att(L, hq=1) == SHAPE
    assert att(L, ldq=248) == SHAPE
    assert att(L, ldy=248) == SHAPE
    assert att(L, window=-1) == SHAPE
    assert att(L, window=1 << 31) == SHAPE
    assert att(L, scale=float("nan")) == UNSUP
    assert att(L, scale=float("inf")) == UNSUP
    assert att(L, cap=-1.0) == UNSUP
    assert att(L, cap=float("inf")) == UNSUP
    assert att(L, q=P + 8) == ALIGN
    assert att(L, y=P + 8) == ALIGN
    assert att(L, ldy=260) == ALIGN
    assert att(L, lse=P + 2) == ALIGN
    assert att(L, slopes=P + 1) == ALIGN
    assert att(L, prefix=P + 2) == ALIGN
    need = L.pdq_kv_attention_workspace(5, 3, 4, 2, 64)
    if need:
        assert att(L, ws=None) == WS
        assert att(L, ws_bytes=need - 1) == WS
        assert att(L, ws=P + 16) == ALIGN


def test_binding_refuses_host_tensors():
    k = torch.zeros((2, 1, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        pdq.KVCache(k, torch.zeros((2, 1, 4, 64, 4), dtype=torch.int8), torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        pdq.KVBatch(torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_oracle_value_layout_round_trip():
    v = np.random.default_rng(0).integers(-127, 128, (3, 2, 32, 64)).astype(np.int8)
    d = KO.device_v(v)
    assert d.shape == (3, 2, 8, 64, 4) and d[1, 1, 2, 5, 3] == v[1, 1, 11, 5]
    assert np.array_equal(KO.plain_v(d), v)


def test_oracle_append_by_hand():
    # one head, page 16: a first token of absmax 127 (scale 1), then one of absmax 254 (scale 2: the held codes halve,
    # ties to even), then one of absmax 1 (the scale stays, the codes are rne(x / 2))
    c = dict(k=np.full((1, 1, 16, 64), 9, np.int8), v=np.full((1, 1, 16, 64), 9, np.int8),
             k_scale=np.full((1, 1), 99, np.float32), v_scale=np.full((1, 1), 99, np.float32))
    table = np.zeros((1, 1), np.int32)

    def one(n, head):
        x = np.zeros((1, 1, 64), np.float32)
        x[0, 0, :4] = head
        KO.append(c, table, [n], None, x, x)

    one(1, [127, 3, -5, 0])
    assert c["k_scale"][0, 0] == 1 and c["k"][0, 0, 0, :4].tolist() == [127, 3, -5, 0] and c["k"][0, 0, 1, 0] == 9
    one(2, [-254, 4, 0, 0])
    assert c["k_scale"][0, 0] == 2
    assert c["k"][0, 0, 0, :4].tolist() == [64, 2, -2, 0]  # 63.5 -> 64, 1.5 -> 2, -2.5 -> -2
    assert c["k"][0, 0, 1, :2].tolist() == [-127, 2] and c["k"][0, 0, 2, 0] == 9
    one(3, [1, -3, 0, 0])
    assert c["k_scale"][0, 0] == 2 and c["k"][0, 0, 2, :2].tolist() == [0, -2]  # 0.5 -> 0, -1.5 -> -2
    one(4, [np.inf, 0, 0, 0])
    assert np.isnan(c["v_scale"][0, 0]) and not c["v"][0, 0, 3].any()


def test_oracle_rotation_keeps_length_and_turns_by_differences():
    half, r = 32, np.random.default_rng(1)
    angle = np.arange(40)[:, None] * 10000.0 ** (-np.arange(half) / half)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    a, b = r.normal(size=(2, 1, 64)).astype(np.float32)
    for inter in (False, True):
        dots = [float((KO.rotate(a, p + 7, cos, sin, inter) * KO.rotate(b, p, cos, sin, inter)).sum()) for p in (0, 9, 30)]
        assert np.allclose(dots, dots[0], atol=64 * 2.0 ** -20)
        assert np.allclose((KO.rotate(a, 33, cos, sin, inter) ** 2).sum(), (a ** 2).sum(), rtol=64 * 2.0 ** -22)
    assert np.isnan(KO.rotate(a, 40, cos, sin, False)).all()
