"""The experts' layer's numerics, each way through it held to what its sums promise (MI355X): sums free of the matrix unit's
alignment for few rows and binary16, the aligned ones of the tiles over many groups, rows that are not finite in every kernel."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from fp8_cases import DT, randn, values
from test_gpu_experts import check, layer
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def unsure(x, r, gate_up, down, sums=2.0 ** -19):
    """What the codes of h may add to y where h lies so near to a border that a sum's last bits decide.

    Gate and up as binary32 sums of exact products: an addition is off by 2^-25 of the sum by chance, some hundred of
    them by less than 2^-21 of the products' root sum of squares; counted four times over, 2^-19 (`sums`).  silu by (1.3 |g| + 7)
    2^-24 (include/pdq.h); its slope is at most 1.1."""
    v, ids, w = FO.values(values(x)), r.ids.cpu().numpy(), values(r.weights)
    slack = np.zeros((v.shape[0], down[1].shape[1]))
    for e in range(r.experts):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        a, b = (gate_up[1][e, i] * FO.spread(gate_up[2][e, i], *gate_up[1].shape[2:]) for i in range(2))
        d = np.abs(down[1][e] * FO.spread(down[2][e], *down[1].shape[1:]))
        gate, up = v[t] @ a.T, v[t] @ b.T
        off = [sums * np.sqrt(v[t] ** 2 @ m.T ** 2) for m in (a, b)]
        h = np.abs(FO.silu_mul(gate, up))
        dh = 1.1 * off[0] * np.abs(up) + np.abs(FO.silu_mul(gate, 1.0)) * off[1] + (1.3 * np.abs(gate) + 8) * 2.0 ** -24 * h
        step = np.abs(FO.values(h + dh) - FO.values(np.maximum(h - dh, 0)))
        np.add.at(slack, t, np.abs(w[t, j, None]) * (step @ d.T))
    return slack


# two launches (tokens * k <= 8), blocks of 16 rows (less than 12 rows an expert), tiles
@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("tokens,experts,k", [(1, 4, 2), (2, 4, 2), (4, 3, 2), (1, 8, 8), (8, 3, 1), (10, 4, 2), (40, 8, 2), (100, 2, 1)])
def test_sums_of_binary16_rows_are_whole(tokens, experts, k, seed, scales):
    """y's rounding, 2^-11 / sqrt(3) at most over all outputs, and the down product's alignment, 2^-12 (fp8_cases.check_linear), in
    quadrature less than 2^-11; and the codes that are unsure.  (With gate and up aligned too the error is 0.0013 = 2.7 * 2^-11.)"""
    gate_up, down = layer(100 * seed + tokens, experts, 1024, 272, scales)
    x = randn(seed + tokens, tokens, 1024).half()
    r = pdq.route_experts(randn(seed + 7, tokens, experts, spread=0.0).cuda(), k)
    y = values(pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"])
    y64, _ = FO.experts(values(x), r.ids.cpu().numpy(), values(r.weights), *gate_up[1:], *down[1:])
    slack = unsure(x, r, gate_up, down)
    assert np.linalg.norm(y - y64) <= 2.0 ** -11 * np.linalg.norm(y64) + np.linalg.norm(slack)


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("tokens,experts,k", [(1, 4, 2), (4, 3, 2), (1, 8, 8), (8, 3, 1), (10, 4, 2), (40, 8, 2), (45, 4, 1)])
def test_few_rows_are_alike_in_both_types(tokens, experts, k, scales):
    """Few rows an expert take the same sums whatever their type: y in bfloat16 and in binary16 are two roundings of one value."""
    gate_up, down = layer(tokens, experts, 1168, 400, scales)
    x = randn(tokens, tokens, 1168).bfloat16()
    x[x.abs() < 2.0 ** -14] = 0
    assert torch.equal(x.half().bfloat16(), x)
    r = pdq.route_experts(randn(tokens + 7, tokens, experts, spread=0.0).cuda(), k)
    a, b = (values(pdq.experts_fp8(v.cuda(), r, gate_up[0], down[0])["y"]) for v in (x, x.half()))
    assert np.all(np.abs(a - b) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(b) + 2.0 ** -24)


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("hidden", [1040, 1168])  # 9 and 10 groups
@pytest.mark.parametrize("tokens,experts,k", [(60, 4, 1), (90, 4, 2), (180, 2, 2), (200, 2, 1), (330, 2, 1)])
def test_tiles_of_bfloat16_rows(tokens, experts, k, hidden, scales):
    """Gate and up in FP8 tiles of 64, 128 and 256 or 192 rows, over more groups than one load of their scales holds.

    Over all outputs.  The aligned sums lose what lies 13 bits behind the largest of eight products: e4m3 products have 8 bits, so
    that only those 2^-6 of it or smaller lose any, a tenth of them (normal factors), 2^-13 of it or less each: of the sum's
    root mean square sqrt(0.1) 2.5 2^-13 / sqrt(3) < 2^-14.  h is off by sqrt(2) 1.5 0.8 of that on average, 1.7 * 2^-14 of
    itself, and passes a border between two codes, 2^-3 to 2^-4 of h apart, with an error of that distance: in the mean of
    squares 1.7 * 2^-14 * 0.7 * 2^-3, 2^-8.4.  y's rounding is 2^-8 / sqrt(3) at most, the down product's alignment 2^-12: in
    quadrature less than 2^-8.
    Of one row, whose norm a single large h may make up half of: a border passed by that one is 2^-3 to 2^-4 of it, up to 2^-4 of
    the row.  So rows are held to y's rounding and alignment, 2^-8, and to their own unsure codes, the sums' error
    counted four times over."""
    gate_up, down = layer(tokens + hidden, experts, hidden, 400, scales)
    x = randn(tokens, tokens, hidden).bfloat16()
    r = pdq.route_experts(randn(tokens + 7, tokens, experts, spread=0.0).cuda(), k)
    y = values(pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"])
    y64, _ = FO.experts(values(x), r.ids.cpu().numpy(), values(r.weights), *gate_up[1:], *down[1:])
    assert np.linalg.norm(y - y64) <= 2.0 ** -8 * np.linalg.norm(y64)
    rows = np.linalg.norm(unsure(x, r, gate_up, down, 2.0 ** -12), axis=1)
    assert np.all(np.linalg.norm(y - y64, axis=1) <= 2.0 ** -8 * np.linalg.norm(y64, axis=1) + rows)


@pytest.mark.parametrize("dt,scales", [("bf16", "pow2"), ("bf16", "f32"), ("f16", "pow2"), ("f16", "f32")])
@pytest.mark.parametrize("tokens,experts,k", [(2, 4, 2), (8, 3, 1), (20, 8, 2), (40, 4, 2), (80, 2, 2), (200, 2, 2)])
def test_rows_that_are_not_finite_stay_alone(tokens, experts, k, dt, scales):
    """In each of the kernels: a row with an infinity or a NaN is NaN, the others are what they are without it."""
    gate_up, down = layer(tokens, experts, 272, 400, scales)
    x = randn(tokens, tokens, 272).to(DT[dt])
    r = pdq.route_experts(randn(tokens + 7, tokens, experts, spread=0.0).cuda(), k)
    y = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"]
    check(y, x, r, gate_up, down)
    bad = {0: (3, float("inf")), tokens // 2: (271, float("nan")), tokens - 1: (130, -float("inf"))}
    for t, (at, v) in bad.items():
        x[t, at] = v
    z = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"]
    rest = [t for t in range(tokens) if t not in bad]
    assert torch.isnan(z[sorted(bad)]).all() and torch.equal(z[rest], y[rest])


@pytest.mark.parametrize("dt,scales", [("bf16", "pow2"), ("f16", "f32")])
def test_tiles_between_the_rules(dt, scales):
    """An average of 160 to 200 rows an expert, unevenly: the largest tiles, partly filled."""
    tokens, experts, k = 175, 4, 4
    gate_up, down = layer(5, experts, 272, 144, scales)
    x = randn(6, tokens, 272).to(DT[dt])
    z = randn(7, tokens, experts, spread=0.0)
    r = pdq.route_experts(z.cuda(), k)
    check(pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"], x, r, gate_up, down)
    z[:, 1:3][torch.randn((tokens, 2), generator=torch.Generator().manual_seed(8)) > 0.5] = -float("inf")
    r = pdq.route_experts(z.cuda(), k)
    check(pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"], x, r, gate_up, down)
