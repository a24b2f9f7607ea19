"""Routing to experts against the oracle (MI355X)."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from fp8_cases import DT, values
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def check(r, logits, k, bias=None, **rule):
    ids, weights, offsets, rows = FO.route(values(logits), k, bias=None if bias is None else values(bias), **rule)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    got = values(r.weights)
    assert np.array_equal(np.isnan(got), np.isnan(weights))
    # binary64 on both sides, one rounding to binary32
    fine = ~np.isnan(weights)
    assert np.all(np.abs(got - weights)[fine] <= np.abs(weights[fine]) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150)


def run(logits, k, bias=None, **rule):
    r = pdq.route_experts(logits.cuda(), k, bias=None if bias is None else bias.cuda(), **rule)
    check(r, logits, k, bias, **rule)
    return r


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 32, 4), (2, 7, 7), (33, 64, 8), (65, 65, 3), (100, 160, 6),
                                              (257, 300, 8), (40, 512, 32), (700, 9, 2)])
def test_softmax(tokens, experts, k, dt):
    run(randn(tokens + experts, tokens, experts).to(DT[dt]), k)
    run(randn(tokens + experts + 1, tokens, experts).to(DT[dt]), k, renormalize=False, scale=2.5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,k,groups,top_groups", [(1, 32, 4, 8, 3), (70, 160, 6, 8, 3), (33, 64, 8, 64, 9),
                                                                (9, 512, 16, 16, 2), (50, 24, 5, 3, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_and_bias(tokens, experts, k, groups, top_groups, score, dt):
    x = randn(experts + k, tokens, experts).to(DT[dt])
    bias = 0.1 * randn(experts, experts)
    for b in (None, bias):
        for group_score in (1, 2):
            run(x, k, b, score=score, groups=groups, top_groups=top_groups, group_score=group_score, scale=1.5)


def test_ties_go_to_the_lowest_index():
    x = torch.zeros((5, 100))
    x[1, 40:] = 1.0
    x[2, ::3] = -2.0
    x[3] = torch.arange(100).flip(0) // 10
    x[4, 70] = -0.0
    run(x, 8)
    run(x, 8, torch.zeros(100), score="sigmoid", groups=10, top_groups=4, group_score=2)


def test_values_that_are_not_numbers():
    inf, nan = float("inf"), float("nan")
    x = randn(1, 9, 70)
    x[0] = -inf                      # nothing to choose
    x[1, 3:] = -inf                  # fewer than k
    x[2, 10] = nan
    x[3] = nan
    x[4, 7] = inf                    # all of a softmax's weight
    x[5, [3, 60]] = inf
    x[6, 5:] = nan
    x[6, :5] = -inf
    x[7] = -1e30
    bias = 0.1 * randn(2, 70)
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for renormalize in (True, False):
                run(x, 6, b, score=score, renormalize=renormalize)
            run(x, 6, b, score=score, groups=7, top_groups=2, group_score=2)
    bias[5] = -inf
    run(randn(3, 20, 70), 6, bias, score="sigmoid")


def test_strided_logits_and_workspace():
    x = randn(4, 40, 128).cuda()
    part = x[:, 3:63]
    r = pdq.route_experts(part, 4, workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda").fill_(0xA5))
    check(r, part.cpu(), 4)


def test_no_tokens():
    r = pdq.route_experts(torch.empty((0, 16), device="cuda"), 2)
    assert r.offsets.cpu().tolist() == [0] * 17 and r.rows.numel() == 0


def test_many_tokens():
    # more workgroups than one, uneven experts
    x = randn(5, 9001, 40) + 2.0 * randn(6, 40)
    ids, weights, offsets, rows = (t.cpu().numpy() for t in (lambda r: (r.ids, r.weights, r.offsets, r.rows))(
        pdq.route_experts(x.cuda(), 3)))
    want = np.argsort(-x.numpy(), 1, kind="stable")[:, :3]
    assert np.array_equal(ids, want)
    o, r = FO.sort_rows(want, 40)
    assert np.array_equal(offsets, o) and np.array_equal(rows, r)
    assert np.all(np.abs(weights.sum(1) - 1) <= 3 * 2.0 ** -24)
