"""Rows of logits whose choices lie within a few steps of fp32, so that the order
of their fp32 values says nothing: the choice is still that of the scores in 64
bits.  (Tolerances: tests/test_gpu_route.py.)"""
import pytest
import torch

import numpy as np

from route_support import DEV
from test_gpu_route import HP, SIG, SOFT, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [64, 100, 128, 250, 256, 512, 600, 1024])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_rows_of_a_few_fp32_steps(experts, score):
    """Scores and biases that move a choice by less than two of its fp32 steps, each
    by its own amount: a row's choices take two or three values in fp32."""
    gen = torch.Generator(device=DEV).manual_seed(experts)
    s = 0.5 if score == SIG else 1.0 / experts
    step = float(np.spacing(np.float32(s)))
    rnd = lambda *shape: torch.rand(*shape, generator=gen, device=DEV)  # noqa: E731
    logits = rnd(30, experts) * (0.1 * step / (s * (1 - s)))
    bias = rnd(experts) * (1.2 * step)
    for topk in (1, 7, 8, 15, 16):
        check(logits, HP(topk, score, 1), bias)
        if experts % 4 == 0:
            check(logits, HP(min(topk, experts // 4), score, 1, 4, 1, 1), bias)
            check(logits, HP(min(topk, experts // 2), score, 1, 4, 2, 2), bias)


@pytest.mark.parametrize("experts", [64, 128, 256, 512, 1024])
def test_two_choices_that_fp32_turns_round(experts):
    """Sigmoids of 1e-8 and 4e-8 with biases of 3.0e-8 and 2.9e-8: 0.5 + 3.25e-8 and
    0.5 + 3.9e-8, in fp32 0.50000006 and 0.5.  The others lie behind both."""
    logits = torch.zeros(5, experts, device=DEV)
    logits[:, 0], logits[:, 1] = 1e-8, 4e-8
    bias = torch.zeros(experts, device=DEV)
    bias[0], bias[1] = 3.0e-8, 2.9e-8
    for topk in (1, 2, 8):
        idx = check(logits, HP(topk, SIG, 1), bias)
        assert bool((idx[:, 0] == 1).all())
