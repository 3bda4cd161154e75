"""Every way that routing takes through its kernels, against the definition in 64
bits: each width of a lane, with all of its experts there or not, up to 8 and 16
choices and more, fours of experts that are one access or not, groups that are
whole lanes or not; rows that have to be chosen again in 64 bits next to rows that
have not, in one wavefront.  (Tolerances: tests/test_gpu_route.py.)"""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, DTYPES, f64, route
from test_gpu_route import HP, SIG, SOFT, check, check_grad, normal, run, run_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts", [16, 60, 63, 64, 100, 128, 130, 252, 256, 260, 509, 512, 516, 1021, 1024])
@pytest.mark.parametrize("topk", [1, 7, 8, 9, 15, 16, 17])
def test_widths(dtype, experts, topk):
    topk = min(topk, experts)
    logits = normal(experts * topk, 21, experts).to(DTYPES[dtype])
    bias = normal(experts, experts, std=0.1)
    check(logits, HP(topk, SOFT, 0))
    check(logits, HP(topk, SIG, 1), bias)
    idx = check(logits, HP(topk, SOFT, 1), bias * 0.01)
    check_grad(logits, HP(topk, SOFT, 0), idx, normal(1, 21, topk))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts", [16, 32, 64, 80, 128, 160, 256, 272, 512, 1024])
@pytest.mark.parametrize("groups", [2, 4, 8, 16])
def test_groups_of_lanes(dtype, experts, groups):
    logits = normal(experts + groups, 45, experts).to(DTYPES[dtype])
    bias = normal(experts, experts, std=0.1)
    for top_groups in (1, groups // 2, groups):
        topk = min(8, experts // groups * top_groups)
        for score in (SOFT, SIG):
            check(logits, HP(topk, score, 1, groups, top_groups, 2), bias)
            check(logits, HP(topk, score, 0, groups, top_groups, 1), bias)
        check(logits, HP(topk, SIG, 1, groups, top_groups, 1))


@pytest.mark.parametrize("experts", [64, 256])
@pytest.mark.parametrize("groups", [1, 8])
def test_rows_chosen_again_beside_others(experts, groups):
    """Of every four neighbouring rows one, another one each time, has choices
    closer than fp32 shows, and one has an infinite bias' expert masked."""
    tokens = 64
    logits = normal(3, tokens, experts)
    near = torch.nextafter(torch.full((), 0.5, device=DEV), torch.full((), 1.0, device=DEV))
    for t in range(tokens):
        if t % 4 == t // 4 % 4:
            logits[t, ::3], logits[t, 1::3], logits[t, 2::3] = 0.5, near, -2.0
        if t % 4 == (t // 4 + 1) % 4:
            logits[t, 5:] = -math.inf
    bias = torch.where(torch.arange(experts, device=DEV) % 2 == 0, 1e-8, 0.0)
    for best in (1, 2) if groups > 1 else (1,):
        for score in (SOFT, SIG):
            hp = HP(6, score, 1, groups, max(1, groups // 2), best)
            check(logits, hp, bias)
            check(logits, hp)
    b = bias.clone()
    b[3] = math.inf
    check(logits, HP(6, SIG, 1, groups, max(1, groups // 2), 1), b)


@pytest.mark.parametrize("spread", [1e-30, 1e-3, 40.0, 1e4, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_spreads(spread, dtype):
    """Logits that nearly agree and logits far apart: the same choice."""
    logits = (normal(17, 40, 256, std=1.0) * spread).to(DTYPES[dtype])
    for topk in (4, 8, 16):
        idx, _ = run(logits, HP(topk, SOFT, 1))
        want, _ = route(f64(logits), None, HP(topk, SOFT, 1))
        assert np.array_equal(idx.cpu().numpy(), want)
        idx, _ = run(logits, HP(topk, SIG, 0), normal(18, 256, std=0.1))
        want, _ = route(f64(logits), f64(normal(18, 256, std=0.1)), HP(topk, SIG, 0))
        assert np.array_equal(idx.cpu().numpy(), want)


def test_equal_rows():
    """A router of zeros: the first experts, each with the same weight."""
    for dtype in DTYPES.values():
        logits = torch.zeros(300, 256, dtype=dtype, device=DEV)
        for score in (SOFT, SIG):
            for bias in (None, torch.zeros(256, device=DEV)):
                idx, w = run(logits, HP(8, score, 1), bias)
                assert bool((idx == torch.arange(8, device=DEV)).all()) and bool((w == 0.125).all())


def test_zeros_of_both_signs_are_one():
    logits = torch.zeros(5, 64, device=DEV)
    logits[:, ::2] = -0.0
    for dtype in DTYPES.values():
        idx, _ = run(logits.to(dtype), HP(4, SOFT, 1))
        assert bool((idx == torch.arange(4, device=DEV)).all())


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 15, 16, 17])
def test_few_tokens_leave_what_lies_behind(tokens):
    logits = normal(tokens, tokens, 64)
    idx = torch.full((tokens + 20, 8), 77, dtype=torch.int32, device=DEV)
    w, d = torch.full((tokens + 20, 8), 77.0, device=DEV), torch.full((tokens + 20, 64), 77.0, device=DEV)
    osa.optim_route(logits, HP(8), idx[:tokens], w[:tokens])
    osa.optim_route_grad(logits, HP(8), idx[:tokens], w[:tokens], d[:tokens])
    assert bool((idx[tokens:] == 77).all()) and bool((w[tokens:] == 77).all()) and bool((d[tokens:] == 77).all())
    assert bool((idx[:tokens] < 64).all()) and torch.equal(d[:tokens], run_grad(logits, HP(8), idx[:tokens], w[:tokens]))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts,topk", [(1, 1), (3, 2), (8, 2), (8, 8), (9, 1), (13, 8), (16, 4)])
def test_many_tokens_of_few_experts(dtype, experts, topk):
    """Large batches of few experts have a kernel of their own: the first and last
    rows against the definition, among them masked ones, infinities and NaN; all
    of them against the same rows in small batches."""
    tokens = 16384 + 37
    logits = normal(experts, tokens, experts).to(DTYPES[dtype])
    logits[3], logits[4, 0], logits[5, experts - 1], logits[6] = -math.inf, math.nan, math.inf, torch.finfo(DTYPES[dtype]).min
    logits[7, 1:], logits[8] = -math.inf, 0.0
    logits[-1, 0] = -math.inf
    bias = normal(99, experts, std=0.1)
    some = torch.cat([torch.arange(40), torch.arange(tokens - 40, tokens)]).to(DEV)
    for hp, b in ((HP(topk, SOFT, 1), None), (HP(topk, SOFT, 0, scale=0.5), None), (HP(topk, SIG, 1), bias), (HP(topk, SOFT, 1), bias),
                  (HP(topk, SIG, 0), None)):
        idx, w = run(logits, hp, b)
        few_idx = check(logits[some].contiguous(), hp, b)
        few_w = run(logits[some].contiguous(), hp, b)[1]
        assert torch.equal(idx[some], few_idx)
        assert torch.allclose(w[some], few_w, rtol=2 * 150 * 2.0 ** -24, atol=1e-37, equal_nan=True)
        parts = [run(logits[a:a + 8000].contiguous(), hp, b)[0] for a in range(0, tokens, 8000)]
        assert torch.equal(idx, torch.cat(parts))
    loose = torch.full((tokens, experts + 3), math.nan, dtype=DTYPES[dtype], device=DEV)
    loose[:, :experts] = logits
    a, b = run(logits, HP(topk)), run(loose[:, :experts], HP(topk))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


@pytest.mark.parametrize("experts,groups", [(64, 1), (256, 8)])
def test_choices_around_the_lowest_place(experts, groups):
    """A bias of 64 for one expert and of 32 for the others: their choices lie where
    a row's places begin, some above and some below by less than fp32 shows."""
    steps = torch.randint(-40, 40, (400, experts), device=DEV, generator=torch.Generator(device=DEV).manual_seed(12)).float()
    logits = 0.3 + steps * 2.0 ** -23
    bias = torch.full((experts,), 32.0, device=DEV)
    bias[5], bias[6] = 64.0, 0.0
    for topk in (2, 3, 8):
        for score in (SIG, SOFT):
            check(logits, HP(topk, score, 1, groups, max(1, groups // 2), 1), bias)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts,groups", [(9, 3), (36, 12), (75, 5), (90, 2), (90, 3), (130, 13), (136, 8), (210, 14), (248, 8), (252, 6),
                                            (340, 17), (504, 8), (1008, 16), (1020, 12), (1023, 3), (1023, 11)])
def test_groups_of_any_size(dtype, experts, groups):
    logits = normal(experts + groups, 37, experts).to(DTYPES[dtype])
    logits[4, :experts // groups] = -math.inf  # a group without any
    logits[5, experts // groups:] = -math.inf  # one group alone
    bias = normal(experts, experts, std=0.1)
    for top_groups in (1, max(1, groups // 2), groups):
        topk = min(8, experts // groups * top_groups)
        for score in (SOFT, SIG):
            check(logits, HP(topk, score, 1, groups, top_groups, 2), bias)
            check(logits, HP(topk, score, 0, groups, top_groups, 1), bias)
        check(logits, HP(topk, SIG, 1, groups, top_groups, 1))
        check(logits, HP(min(16, experts // groups * top_groups), SOFT, 1, groups, top_groups, 1))


@pytest.mark.parametrize("experts,topk", [(12, 5), (64, 6), (64, 8), (256, 8), (256, 16), (300, 8)])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_logits_that_passed_through_16_bits(experts, topk, score):
    """Many equal logits in fp32 and in bf16, without a bias, with none so far and
    with one of a few levels; among them rows with a choice nearly equal to others."""
    logits = normal(31, 60, experts).to(torch.bfloat16).float()
    logits[::4] = logits[::4].round()
    logits[1::8, 3] = torch.nextafter(logits[1::8, 2], torch.full((), 9.0, device=DEV))
    logits[5, 4:] = -math.inf
    levels = torch.randint(-2, 3, (experts,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).float() * 1e-3
    for bias in (None, torch.zeros(experts, device=DEV), levels):
        check(logits, HP(topk, score, 1), bias)
        check(logits.to(torch.bfloat16), HP(topk, score, 0), bias)
        if experts % 4 == 0:
            check(logits, HP(min(topk, experts // 2), score, 1, 4, 2, 1), bias)
