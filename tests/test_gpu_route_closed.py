"""What routing's gradient gives experts that are not open: nothing where the
logit shuts them, and their softmax' share where only the bias does, which is in
the choice but not in the scores.  (Tolerances: tests/test_gpu_route.py.)"""
import math

import pytest
import torch

from route_support import DEV, DTYPES
from test_gpu_route import HP, SIG, SOFT, check, check_grad, normal, run_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts,topk", [(12, 3), (64, 8), (256, 8), (512, 20)])
def test_closed_by_the_logit_and_closed_by_the_bias(dtype, experts, topk):
    logits, bias, dw = normal(1, 20, experts).to(DTYPES[dtype]), normal(2, experts, std=0.1), normal(3, 20, topk)
    logits[:, 2], logits[::2, 4] = -math.inf, math.nan
    bias[1], bias[3] = -math.inf, math.nan
    for score in (SOFT, SIG):
        for renormalise in (0, 1):
            hp = HP(topk, score, renormalise)
            idx = check(logits, hp, bias)
            assert not bool(((idx == 1) | (idx == 2) | (idx == 3)).any()) and not bool((idx[::2] == 4).any())
            # (a NaN logit's weights are NaN, which have no derivative: as closed by -inf)
            check_grad(torch.nan_to_num(logits, nan=-math.inf, neginf=-math.inf), hp, idx, dw)
            d = run_grad(logits, hp, idx, dw)
            assert torch.equal(d, run_grad(torch.nan_to_num(logits, nan=-math.inf, neginf=-math.inf), hp, idx, dw))
            assert bool((d[:, 2] == 0).all()) and bool((d[::2, 4] == 0).all())
            whole = score == SOFT and not renormalise
            assert bool((d[:, [1, 3]] != 0).any()) == whole
