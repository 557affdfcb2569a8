"""Selections and their gradient at the ends of fp32's range, against the
definition in 64 bits."""

import math

import pytest
import torch

from tests.test_gpu_select import check

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


def logits_of(T, E, seed=0):
    return torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("kept", [1, 2, 3, 4, 5])
def test_groups_switched_off_by_the_types_lowest_value(score, best, kept):
    """Biases of fp32's lowest value add up to more than fp32 holds; such a group
    still comes before one whose experts have -inf."""
    T, E, G = 70, 48, 6
    bias = torch.zeros((G, E // G), device="cuda")
    bias[0] = -math.inf
    bias[1] = LOW
    bias[2] = -1e38
    bias[2, 1] = LOW
    bias[3, 1:] = LOW
    bias[4] = LOW
    bias[4, 3] = -3e38
    k = min(16, kept * E // G)
    check(T, E, k, (score, G, kept, best, True, 0.0), logits=logits_of(T, E), bias=bias.view(-1))
    bias[5] = LOW
    check(T, E, k, (score, G, kept, best, False, 0.0), logits=logits_of(T, E, 1), bias=bias.view(-1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kept", [1, 2, 4])
def test_groups_of_the_largest_biases(score, kept):
    """Sums of two finite keys beyond fp32's largest number, behind a group with an
    infinite one, in their order."""
    T, E, G = 50, 40, 5
    bias = torch.zeros((G, E // G), device="cuda")
    bias[0, :2] = 2e38
    bias[1, :2] = 3e38
    bias[2, :2] = -LOW
    bias[4, 5] = math.inf
    idx, _ = check(T, E, 8, (score, G, kept, 2, True, 0.0), logits=logits_of(T, E, 2), bias=bias.view(-1))
    assert (idx == 37).any(1).all()
