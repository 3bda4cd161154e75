"""The gradient of weights that sum to scale where one of them has nearly all of
it.  (Formulas and tolerances: tests/test_gpu_route_grad_dominant.py.)"""
import pytest
import torch

from route_support import DEV, DTYPES
from test_gpu_route import HP, SIG, SOFT, normal, run_grad
from test_gpu_route_grad_dominant import check, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts", [48, 256, 1000])
@pytest.mark.parametrize("topk", [1, 2, 8, 16, 20])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_of_renormalised_weights(dtype, experts, topk, score):
    logits, idx, dw = rows(experts, dtype, topk)
    if score == SIG:  # far below zero sigmoids are as far apart as exponentials
        logits = (logits.float() - 30.0).to(DTYPES[dtype])
    check(logits, HP(topk, score, 1, scale=1.5), idx, dw)


@pytest.mark.parametrize("score", [SOFT, SIG])
def test_one_weight_has_no_gradient(score):
    """A weight alone is scale, whatever the logits."""
    logits = normal(3, 20, 64)
    idx = torch.randint(0, 64, (20, 1), device=DEV, dtype=torch.int32)
    assert float(run_grad(logits, HP(1, score, 1, scale=2.0), idx, normal(4, 20, 1)).abs().max()) == 0.0
