"""Balance biases at the ends of fp32's range: masks of the lowest value, of which
two add up to less than any float, and infinities beside the largest float.
(Tolerances: tests/test_gpu_route.py.)"""
import math

import pytest
import torch

from route_support import DEV
from test_gpu_route import HP, SIG, SOFT, check, normal

pytestmark = pytest.mark.gpu
LARGEST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("experts,groups", [(16, 4), (64, 4), (96, 3), (256, 8), (272, 16), (1024, 8)])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_groups_whose_sum_passes_the_lowest_float(experts, groups, score):
    """Every bias is the lowest float, or in some groups: a group of such experts is
    one like others, behind those with larger ones, and not one without any."""
    per = experts // groups
    logits = torch.zeros(12, experts, device=DEV)
    logits[1, :per - 1] = -math.inf             # the first group has one left
    logits[2, :per] = -math.inf                 # and here none
    logits[3, 1:per:2] = -math.inf
    logits[4, per - 1:] = -math.inf             # most experts are not open at all
    logits[5:] = normal(experts, 7, experts)
    logits[6, ::2] = -math.inf
    bias = torch.full((experts,), -LARGEST, device=DEV)
    some = bias.clone()
    some[:per], some[2 * per:] = 0.0, 0.1
    some[3 * per - 1] = -LARGEST
    for b in (bias, some):
        for top_groups in (1, 2):
            for topk in (2, min(8, per)):
                check(logits, HP(topk, score, 1, groups, top_groups, 2), b)
                check(logits, HP(topk, score, 1, groups, top_groups, 1), b)


@pytest.mark.parametrize("experts", [12, 64, 256, 1000])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_an_infinite_bias_is_above_the_largest(experts, score):
    """Of experts with one logit and biases of the largest float and of infinity,
    the infinite ones come first."""
    logits = torch.zeros(6, experts, device=DEV)
    logits[3:] = normal(5, 3, experts)
    bias = torch.zeros(experts, device=DEV)
    bias[3] = bias[9] = LARGEST
    bias[7] = math.inf
    for topk in (1, 2, 4, 8):
        idx = check(logits, HP(topk, score, 1), bias)
        assert bool((idx[:, 0] == 7).all())
    most = torch.full((experts,), LARGEST, device=DEV)
    most[7] = math.inf  # (no expert far below the others)
    for topk in (1, 2, 8):
        assert bool((check(logits, HP(topk, score, 1), most)[:, 0] == 7).all())
    bias[2] = math.inf
    for topk in (1, 2, 4, 8):
        check(logits, HP(topk, score, 1), bias)
        if experts % 4 == 0:
            check(logits, HP(min(topk, experts // 4), score, 1, 4, 1, 1), bias)
            check(logits, HP(min(topk, experts // 4), score, 1, 4, 1, 2), bias)
