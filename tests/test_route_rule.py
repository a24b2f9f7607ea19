"""The routing rule that the binding hands over: the values of the call, whatever objects hold them (no GPU)."""
import pytest
import torch

from w8a8_int8_quantized_absmax_amd import pdq


def rule(score="softmax", k=2, groups=1, top_groups=1, group_score=1, renormalize=True, scale=1.0):
    c = pdq._route_rule(score, k, groups, top_groups, group_score, renormalize, scale)[0]
    return c.score, c.k, c.groups, c.top_groups, c.group_score, c.renormalize, c.scale


def test_a_value_that_changed():
    scale, groups, renormalize = torch.tensor(2.5), torch.tensor(2), torch.tensor(True)
    assert rule(scale=scale, groups=groups, renormalize=renormalize) == (0, 2, 2, 1, 1, 1, 2.5)
    scale.fill_(1.0), groups.fill_(4), renormalize.fill_(False)
    assert rule(scale=scale, groups=groups, renormalize=renormalize) == (0, 2, 4, 1, 1, 0, 1.0)


@pytest.mark.parametrize("name", ["k", "groups", "top_groups", "group_score"])
def test_no_field_wraps(name):
    assert rule(**{name: 2 ** 31 - 1})
    for v in (2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            rule(**{name: v})
    with pytest.raises(TypeError):
        rule(**{name: 1.5})


def test_values_of_other_types():
    assert rule(scale=2) == rule(scale=2.0) == rule(scale=torch.tensor(2.0, dtype=torch.float64))
    assert rule(renormalize=0) == rule(renormalize=False) and rule(renormalize=7)[5] == 1
    assert rule(k=True)[1] == 1
    with pytest.raises(ValueError):
        rule(score="max")
