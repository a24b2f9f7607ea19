"""FP8 products at the ends of the types' ranges (MI355X): wherever the result is inside, it is what the oracle says."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from fp8_cases import DT, check_linear, randn, values, weight
from test_gpu_experts import check
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def scaled(packed, by):
    """A weight's codes with their block scales times `by` (powers of two) -> what fp8_cases.weight returns."""
    s = packed.scales() * by
    packed = pdq.pack_weight_fp8(packed.codes(), (s if packed.scale_type == pdq.SCALE_F32 else s.to(torch.float8_e8m0fnu)).contiguous())
    return packed, packed.codes().cpu().double().numpy(), packed.scales().cpu().double().numpy()


# one size for each kernel: coded within, 16, 32 and 64 rows, the tiles
KERNELS = [(1, 300, 400, 0), (13, 70, 400, 0), (16, 150, 1168, 0), (20, 150, 528, 0), (64, 150, 400, 0), (1030, 4100, 144, 128),
           (1529, 8190, 400, None)]


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("up,down", [(118, -30), (126, -140), (90, -100), (-110, 100), (-126, 30)])
@pytest.mark.parametrize("m,n,k,tile", KERNELS)
def test_linear(m, n, k, tile, up, down, scales):
    """Rows of some 2^up by weights of some 2^down: a row's scale times the sum of codes alone may pass 2^128, or the
    weight's scale lie below 2^-126, where the result is neither."""
    if scales == "pow2":
        down = max(down, -110)  # (the format's smallest is 2^-127)
    x = randn(m + n, m, k).clamp(-3.5, 3.5) * 2.0 ** up
    x[:, :128] *= 2.0 ** -20
    x = x.bfloat16()
    w, wq, ws = scaled(weight(n + k, (), n, k, scales)[0], 2.0 ** down)
    if tile is not None:
        assert pdq.gemm_fp8_tile(m, n, k, w.scale_type) == tile or scales == "pow2"
    rows = np.unique(np.concatenate([np.arange(0, m, max(1, m // 7)), [m - 1]]))
    cols = np.unique(np.concatenate([np.arange(0, n, max(1, n // 60)), np.arange(max(0, n - 20), n)]))
    y = pdq.linear_fp8(x.cuda(), w)["y"][torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
    y64, size, aligned = FO.linear(values(x[rows]), wq, ws)
    pick = np.ix_(np.arange(len(rows)), cols)
    assert np.abs(y64[pick]).max() < 2.0 ** 127
    check_linear(y, y64[pick], size[pick], aligned[pick], k)


def test_scales_of_any_value():
    """Negative, zero, infinite and NaN binary32 scales count as they are."""
    n, k = 400, 272
    for m in (3, 40):
        w, wq, ws = weight(m, (), n, k, "f32")
        s = w.scales()
        s[0, 1], s[1, 0], s[2, 2], s[3, 1] = -0.75, 0.0, float("inf"), float("nan")
        w = pdq.pack_weight_fp8(w.codes(), s.contiguous())
        x = randn(m, m, k).bfloat16()
        y = pdq.linear_fp8(x.cuda(), w)["y"]
        y64, size, aligned = FO.linear(values(x), wq[:256], s[:2].cpu().double().numpy())
        check_linear(y[:, :256], y64, size, aligned, k)
        last = FO.values(values(x))[:, 256:] @ wq[256:384, 256:].T  # the sums of the infinite scale's group
        assert np.array_equal(np.sign(last[last != 0]) * np.inf, values(y[:, 256:384])[last != 0])
        assert torch.isnan(y[:, 384:]).all()


# sizes for each way through the layer: two launches, blocks of 16 rows, tiles of 64, 128 and 256 or 192 rows
@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("tokens,experts,k", [(1, 4, 2), (4, 2, 2), (20, 8, 2), (40, 4, 2), (60, 2, 2), (200, 2, 2)])
def test_experts(tokens, experts, k, scales):
    """x and h of some 2^118, brought back by the weights' scales."""
    hidden, inner = 400, 272
    gate_up = weight(tokens, (experts, 2), inner, hidden, scales)[0]
    by = torch.tensor([2.0 ** -118, 1.0], device="cuda").view(1, 2, 1, 1)
    gate_up = scaled(gate_up, by)
    down = scaled(weight(tokens + 1, (experts,), hidden, inner, scales)[0], 2.0 ** -100)
    x = (randn(tokens + 2, tokens, hidden).clamp(-3.5, 3.5) * 2.0 ** 118).bfloat16()
    r = pdq.route_experts(randn(tokens + 3, tokens, experts, spread=0.0).cuda(), k)
    y = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"]
    check(y, x, r, gate_up, down)


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("dt,up,by", [("bf16", 125, 40), ("f16", 13, 126)])
@pytest.mark.parametrize("tokens,experts,k", [(1, 4, 2), (4, 2, 2), (20, 8, 2), (40, 4, 2), (200, 2, 2), (400, 2, 2)])
def test_blocks_of_zeros(tokens, experts, k, dt, up, by, scales):
    """Blocks of zero codes under a scale that passes 2^128 with the rows': they add nothing."""
    hidden, inner = 400, 272
    g = weight(tokens, (experts, 2), inner, hidden, scales)[0]
    codes, s = g.codes(), g.scales()
    codes.view(torch.uint8)[..., 128:256] = 0
    s[..., 1] = 2.0 ** by
    s[:, :, :, [0, 2, 3]] *= 2.0 ** -up
    g = pdq.pack_weight_fp8(codes, (s if scales == "f32" else s.to(torch.float8_e8m0fnu)).contiguous())
    gate_up = g, g.codes().cpu().double().numpy(), g.scales().cpu().double().numpy()
    down = weight(tokens + 1, (experts,), hidden, inner, scales)
    x = (randn(tokens + 2, tokens, hidden).clamp(-3.5, 3.5) * 2.0 ** up).to(DT[dt])
    r = pdq.route_experts(randn(tokens + 3, tokens, experts, spread=0.0).cuda(), k)
    y = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"]
    check(y, x, r, gate_up, down)
