"""The experts' layer against the oracle (MI355X)."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from fp8_cases import DT, randn, values, weight
from guards import gapped
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def check(y, x, r, gate_up, down):
    """y's rounding; the products' own error (fp8_cases.check_linear: 8 * 2^-13 of the sum of magnitudes at
    most); and h's codes: where h lies next to a border between two of them, the last bits of gate and up decide, and
    the code is a step, 2^-3 of it at most, off.
    Over all outputs: gate and up are off by 2^-12.5 of their size (there), h by sqrt(2) 1.5 times that, 2^-11.4;
    a border is crossed where h is nearer to it than that, with steps of 2^-3 of a binade by chance 0.8 * 2^-11.4 *
    1.44 / 2^-3 = 2^-8.2 of the time, for an error of 2^-3 / 1.44 of h: 2^(-8.2 / 2) 2^-3.5 < 2^-7 of y's size."""
    y64, size = FO.experts(values(x), r.ids.cpu().numpy(), values(r.weights), *gate_up[1:], *down[1:])
    half = torch.finfo(y.dtype).eps / 2
    got = values(y)
    assert np.all(np.abs(got - y64) <= half * np.abs(y64) + (1 + half) * (2.0 ** -3 + 2.0 ** -9) * size)
    assert np.linalg.norm(got - y64) <= (half + 2.0 ** -7) * np.linalg.norm(y64)


def layer(seed, experts, hidden, inner, scales):
    return weight(seed, (experts, 2), inner, hidden, scales), weight(seed + 1, (experts,), hidden, inner, scales)


SIZES = [(1, 1, 1, 16, 16), (1, 8, 3, 256, 128), (2, 4, 4, 144, 272), (5, 6, 2, 512, 144), (37, 5, 2, 272, 256),
         (70, 64, 6, 128, 160), (150, 3, 1, 144, 400), (200, 4, 2, 400, 512)]


@pytest.mark.parametrize("dt,scales", [("bf16", "pow2"), ("f16", "f32")])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", SIZES)
def test_experts(tokens, experts, k, hidden, inner, dt, scales):
    gate_up, down = layer(tokens + experts, experts, hidden, inner, scales)
    x = randn(tokens, tokens, hidden).to(DT[dt])
    r = pdq.route_experts(randn(experts, tokens, experts, spread=0.0).cuda(), k, score="sigmoid", scale=1.5)
    y, untouched = gapped(tokens, hidden, DT[dt])
    out = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0], out=y)["y"]
    untouched()
    check(out, x, r, gate_up, down)
    ws = torch.full((pdq.experts_fp8_workspace_bytes(tokens, k, experts, hidden, inner),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    again = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0], workspace=ws)["y"]
    assert torch.equal(again, out)  # whatever the workspace holds, the same on every call


def test_all_tokens_at_one_expert_and_rows_without():
    experts, hidden, inner = 6, 256, 144
    gate_up, down = layer(3, experts, hidden, inner, "pow2")
    x = randn(7, 40, hidden).bfloat16()
    z = torch.full((40, experts), -float("inf"))
    z[:35, 4] = 1.0                 # rows 35 .. 39 see no expert
    z[::2, 1] = torch.where(torch.arange(20) < 18, 0.5, -float("inf"))
    r = pdq.route_experts(z.cuda(), 3)
    y = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"]
    check(y, x, r, gate_up, down)
    assert (y[36:] == 0).all()
    assert (r.ids[35:].cpu()[1::2] == -1).all()


def test_a_row_of_nan_stays_alone():
    gate_up, down = layer(5, 4, 256, 128, "f32")
    x = randn(8, 30, 256).bfloat16()
    x[11, 3] = float("inf")
    r = pdq.route_experts(randn(9, 30, 4).cuda(), 2)
    y = pdq.experts_fp8(x.cuda(), r, gate_up[0], down[0])["y"].cpu()
    assert torch.isnan(y[11]).all() and torch.isfinite(y[[i for i in range(30) if i != 11]]).all()


def test_entries_that_are_no_rows_are_passed_over():
    gate_up, down = layer(6, 4, 128, 128, "pow2")
    x = randn(10, 20, 128).bfloat16()
    r = pdq.route_experts(randn(11, 20, 4).cuda(), 2)
    ids = r.ids.clone()
    ids[3, 0], ids[4, 1] = -7, 99   # passed over by the sum
    offsets = r.offsets.clone()
    offsets[-1] = 1 << 30
    bad = pdq.Routing(ids, r.weights, offsets, r.rows)
    y = pdq.experts_fp8(x.cuda(), bad, gate_up[0], down[0])["y"]
    keep = pdq.Routing(torch.where((ids >= 0) & (ids < 4), ids, -1), r.weights, r.offsets, r.rows)
    check(y, x, keep, gate_up, down)


def test_no_tokens():
    gate_up, down = layer(6, 2, 128, 128, "pow2")
    r = pdq.route_experts(torch.empty((0, 2), device="cuda"), 1)
    assert pdq.experts_fp8(torch.empty((0, 128), dtype=torch.float16, device="cuda"), r, gate_up[0], down[0])["y"].shape == (0, 128)
