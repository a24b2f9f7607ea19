"""Refusals of the FP8, routing and experts entry points (host checks: nothing is enqueued, no pointer is followed), and
pins of the oracle."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from w8a8_int8_quantized_absmax_amd import pdq

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = range(7)
P = 1 << 20  # an address that is aligned and never read


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pdq.LIB_PATH):
        pytest.skip("libpdq.so not built")
    return pdq.lib()


def test_sizes(L):
    assert L.pdq_fp8_bytes(1, 16) == 16 * 128 and L.pdq_fp8_bytes(17, 129) == 32 * 256
    assert L.pdq_fp8_bytes(0, 64) == 0 and L.pdq_fp8_bytes(-1, 64) == 0
    assert [L.pdq_fp8_scale_pitch(k) for k in (16, 512, 513, 4096)] == [4, 4, 8, 32]
    assert L.pdq_route_workspace(0, 8) == 0 and L.pdq_route_workspace(4, 513) == 0 and L.pdq_route_workspace(1, 8) >= 32
    assert L.pdq_experts_fp8_workspace(4, 2, 8, 256, 100) == 0 and L.pdq_experts_fp8_workspace(4, 2, 8, 256, 128) > 0


def test_quantize_weight(L):
    def f(w=P, dt=1, count=1, n=4, k=32, ld=32, stride=128, wq=P, ws=P):
        return L.pdq_quantize_weight_fp8(w, dt, count, n, k, ld, stride, wq, ws, None)
    assert f(dt=3) == DTYPE
    assert f(k=17, ld=32) == SHAPE and f(ld=16) == SHAPE and f(n=-1) == SHAPE and f(count=-1) == SHAPE
    assert f(count=2, stride=127) == SHAPE and f(count=1 << 21, n=1 << 21) == SHAPE
    assert f(w=None) == NULL and f(wq=None) == NULL and f(ws=None) == NULL
    assert f(w=P + 8) == ALIGN and f(ld=36) == ALIGN and f(wq=P + 4) == ALIGN and f(count=2, stride=132) == ALIGN
    assert f(n=0) == OK and f(count=0) == OK


def test_pack_weight(L):
    def f(c=P, s=P, st=0, count=1, n=4, k=32, wq=P, ws=P):
        return L.pdq_pack_weight_fp8(c, s, st, count, n, k, wq, ws, None)
    assert f(st=2) == DTYPE and f(st=-1) == DTYPE
    assert f(k=24) == SHAPE and f(count=-1) == SHAPE
    assert f(c=None) == NULL and f(s=None) == NULL and f(wq=None) == NULL and f(ws=None) == NULL
    assert f(c=P + 8) == ALIGN and f(st=1, s=P + 2) == ALIGN and f(wq=P + 8) == ALIGN
    assert f(n=0) == OK


def test_linear(L):
    def f(x=P, dt=1, m=400, k=64, ld=64, wq=P, ws=P, st=0, b=None, n=16, y=P, ydt=1, ldy=16, work=P, size=1 << 20):
        return L.pdq_linear_fp8(x, dt, m, k, ld, wq, ws, st, b, n, y, ydt, ldy, work, size, None)
    assert f(dt=3) == DTYPE and f(ydt=0) == DTYPE and f(st=7) == DTYPE
    assert f(k=40, ld=40) == SHAPE and f(k=0) == SHAPE and f(ld=32) == SHAPE and f(ldy=15) == SHAPE and f(n=-1) == SHAPE
    assert f(m=(1 << 21) + 1) == SHAPE and f(k=65552, ld=65552) == SHAPE
    for a in ("x", "wq", "ws", "y"):
        assert f(**{a: None}) == NULL
    for a, by in (("x", 8), ("wq", 8), ("ws", 8), ("y", 1), ("b", 2), ("work", 64)):
        assert f(**{a: P + by}) == ALIGN
    assert f(ld=68) == ALIGN
    assert f(work=None) == WS and f(size=100) == WS
    assert f(m=0) == OK and f(n=0) == OK
    assert L.pdq_linear_fp8_workspace(400, 64) >= L.pdq_fp8_bytes(400, 64) + 400 * L.pdq_fp8_scale_pitch(64)
    assert [L.pdq_linear_fp8_workspace(m, k) for m, k in ((1, 4096), (0, 64), (-1, 64), (4, 60))] == [0] * 4


def test_gemm_tile(L):
    f = L.pdq_gemm_fp8_tile
    assert f(0, 8, 64, 0) == -1 and f(8, 0, 64, 0) == -1 and f(8, 8, 0, 0) == -1 and f(8, 8, 64, 5) == -1
    assert f(64, 28672, 4096, 0) == 0 and f(8192, 8192, 4096, 0) == 256 and f(8192, 8192, 4096, 1) in (128, 192)


def test_gemm_and_quantize(L):
    assert L.pdq_gemm_fp8(P, P, 0, 64, P, P, 0, None, 16, P, 1, 16, None) == OK
    assert L.pdq_gemm_fp8(P, P, 4, 64, P, P, 0, None, 0, P, 1, 16, None) == OK
    assert L.pdq_gemm_fp8(P, P, 4, 63, P, P, 0, None, 16, P, 1, 16, None) == SHAPE
    assert L.pdq_gemm_fp8(None, P, 4, 64, P, P, 0, None, 16, P, 1, 16, None) == NULL
    assert L.pdq_gemm_fp8(P, None, 4, 64, P, P, 0, None, 16, P, 1, 16, None) == NULL
    assert L.pdq_gemm_fp8(P + 8, P, 4, 64, P, P, 0, None, 16, P, 1, 16, None) == ALIGN
    assert L.pdq_gemm_fp8(P, P + 2, 4, 64, P, P, 0, None, 16, P, 1, 16, None) == ALIGN
    assert L.pdq_quantize_fp8(P, 1, 0, 64, 64, P, P, None) == OK
    assert L.pdq_quantize_fp8(P, 1, 4, 64, 64, None, P, None) == NULL
    assert L.pdq_quantize_fp8(P, 1, 4, 64, 64, P + 8, P, None) == ALIGN


def test_product_limit(L):
    # 2^38 outputs; the pointers are followed by no one, as the bias is misaligned
    def f(m, n):
        return L.pdq_gemm_fp8(P, P, m, 16, P, P, 0, P + 2, n, P, 1, n, None)
    assert f(1 << 21, 1 << 17) == ALIGN and f(1 << 21, (1 << 17) + 1) == SHAPE


def test_route(L):
    def f(x=P, dt=0, t=4, e=16, ld=16, b=None, score=0, k=2, g=1, tg=1, gs=1, renorm=1, scale=1.0, ids=P, w=P, o=P, r=P,
          ws=P, size=1 << 20, rule=True):
        c = pdq._RouteRuleC(score, k, g, tg, gs, renorm, scale)
        return L.pdq_route_experts(x, dt, t, e, ld, b, ctypes.byref(c) if rule else None, ids, w, o, r, ws, size, None)
    assert f(dt=3) == DTYPE and f(rule=False) == NULL
    assert f(e=0) == SHAPE and f(e=513, ld=513) == SHAPE and f(ld=15) == SHAPE and f(t=-1) == SHAPE
    assert f(k=0) == SHAPE and f(k=17) == SHAPE and f(k=33, e=64, ld=64) == SHAPE
    assert f(g=3) == SHAPE and f(g=0) == SHAPE and f(g=128, e=128, ld=128) == SHAPE and f(g=4, tg=5) == SHAPE and f(tg=0) == SHAPE
    assert f(score=2) == UNSUP and f(gs=0) == UNSUP and f(gs=3) == UNSUP and f(scale=float("nan")) == UNSUP
    for a in ("x", "ids", "w", "o", "r"):
        assert f(**{a: None}) == NULL
    assert f(x=P + 2) == ALIGN and f(b=P + 2) == ALIGN and f(ids=P + 2) == ALIGN and f(ws=P + 64) == ALIGN
    assert f(ws=None) == WS and f(size=0) == WS


def test_experts(L):
    def f(x=P, dt=1, ld=64, t=4, e=8, k=2, h=64, i=32, st=0, gu=P, gus=P, d=P, ds=P, ids=P, w=P, o=P, r=P, re=None, y=P,
          ldy=64, ws=P, size=1 << 30, routing=True, experts=True):
        a = pdq._RoutingC(ids, w, o, r, t, e if re is None else re, k)
        b = pdq._ExpertsC(gu, gus, d, ds, st, e, h, i)
        return L.pdq_experts_fp8(x, dt, ld, ctypes.byref(a) if routing else None, ctypes.byref(b) if experts else None, y, ldy,
                                 ws, size, None)
    assert f(dt=0) == DTYPE and f(st=5) == DTYPE and f(routing=False) == NULL and f(experts=False) == NULL
    assert f(h=40) == SHAPE and f(i=24) == SHAPE and f(k=9) == SHAPE and f(re=7) == SHAPE and f(e=513) == SHAPE
    assert f(ld=48) == SHAPE and f(ldy=60) == SHAPE and f(t=-1) == SHAPE and f(t=1 << 21, k=8, h=65536, i=65536) == SHAPE
    for a in ("x", "gu", "gus", "d", "ds", "ids", "w", "o", "r", "y"):
        assert f(**{a: None}) == NULL
    assert f(x=P + 8) == ALIGN and f(ld=68) == ALIGN and f(ldy=66) == ALIGN and f(gu=P + 8) == ALIGN and f(ds=P + 8) == ALIGN
    assert f(ws=None) == WS and f(size=100) == WS and f(ws=P + 64) == ALIGN
    assert f(t=0) == OK


def test_oracle_codes_are_e4m3():
    # every e4m3 value is its own code, what lies between goes to the nearest, ties to even (torch's conversion)
    b = np.array([v for v in range(256) if v & 0x7f != 0x7f], np.uint8)
    v = torch.from_numpy(b.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(FO.e4m3(v), v) and np.array_equal(FO.e4m3_bits(v), b)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.exp(3 * torch.randn(20000, generator=torch.Generator().manual_seed(2)))
    mid = torch.from_numpy(np.concatenate([(v[:-1] + v[1:]) / 2, v * (1 + 2.0 ** -20)])).float()
    x = torch.cat([x, mid]).clamp(-448, 448)
    assert np.array_equal(FO.e4m3(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_oracle_scales_are_the_smallest():
    top = np.exp(np.random.default_rng(1).uniform(-80, 85, 4000)).astype(np.float32).astype(np.float64)
    top = np.concatenate([top, 448 * 2.0 ** np.arange(-100, 100), np.nextafter(np.float32(448), np.float32(500)) * 2.0 ** np.arange(-100, 100)])
    s = FO.scale_value(FO.scale_byte(top))
    assert np.all(top <= 448 * s) and np.all(top > 224 * s)
    assert FO.scale_byte([0.0, np.inf, np.nan]).tolist() == [127, 255, 255]


def test_oracle_route_small():
    z = np.array([[1.0, 3.0, 2.0, 3.0]])
    ids, w, o, r = FO.route(z, 2)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, 0.5) and o.tolist() == [0, 0, 1, 1, 2] and r.tolist() == [0, 1]
    ids, w, _, _ = FO.route(z, 2, score="sigmoid", bias=np.array([5.0, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 1 / (1 + np.exp(-z[0, [0, 1]])))
    ids, _, _, _ = FO.route(z, 1, groups=2, top_groups=1, group_score=2)
    assert ids.tolist() == [[3]]


def test_oracle_experts_small():
    x = np.eye(2, 16) * 4
    gu = np.ones((1, 2, 16, 16))
    d = np.ones((1, 16, 16))
    one = np.ones((1, 2, 1, 1))
    y, _ = FO.experts(x, np.array([[0], [-1]]), np.array([[0.5], [0.0]]), gu, one, d, one[:, 0])
    h = FO.values(np.full((1, 16), FO.silu_mul(4.0, 4.0)))[0]
    assert np.allclose(y[0], 0.5 * h.sum()) and not y[1].any()


def test_binding_refuses_host_tensors():
    x, z = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 8))
    ids, rows = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: pdq.quantize_weight_fp8(x), lambda: pdq.quantize_fp8(x), lambda: pdq.linear_fp8(x, None),
                 lambda: pdq.pack_weight_fp8(x.to(torch.float8_e4m3fn), torch.ones((1, 1))),
                 lambda: pdq.route_experts(z, 2), lambda: pdq.experts_fp8(x, None, None, None),
                 lambda: pdq.Routing(ids, torch.zeros((4, 2)), torch.zeros(9, dtype=torch.int32), rows)):
        with pytest.raises(ValueError):
            call()
