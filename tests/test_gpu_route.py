"""Routing to experts and its gradient against the definitions in 64 bits: sizes
from one token and one expert on, both scores, groups, bias, equal logits, rows
without any open expert, infinities, NaN and the types' lowest values, rows that
lie apart.

The choice has to be the 64-bit one.  Weights: exp of a difference x is off by
|x| 2^-24 (the difference's rounding) beside a few steps of 2^-24, a sum of n
positive terms by less than (n / 64 + 6) 2^-24 of itself, and a weight has two
roundings and a quotient: (|x| + 64) 2^-24 of itself covers them.  The
gradient's terms have the same error relative to the largest |g| s of the row,
two of them to each element, and one rounding to the logits' type."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, DTYPES, HALF_STEP, apart, f64, route, route_grad, scores, spread, weights_of

pytestmark = pytest.mark.gpu

HP = osa.optim_route_hp
SOFT, SIG = osa.OPTIM_ROUTE_SOFTMAX, osa.OPTIM_ROUTE_SIGMOID


def run(logits, hp, bias=None):
    idx = torch.full((logits.size(0), hp.topk), -7, dtype=torch.int32, device=DEV)
    w = torch.full((logits.size(0), hp.topk), -7.0, device=DEV)
    osa.optim_route(logits, hp, idx, w, bias=bias)
    torch.cuda.synchronize()
    return idx, w


def run_grad(logits, hp, idx, dw):
    d = torch.full_like(logits, 77.0) if logits.is_contiguous() else apart(*logits.shape, logits.dtype, 3, fill=77.0)[1]
    osa.optim_route_grad(logits, hp, idx, dw, d)
    torch.cuda.synchronize()
    return d


def reach(logits):
    fine = np.where(np.isfinite(logits), logits, 0.0)
    return float(fine.max() - fine.min()) if fine.size else 0.0


def check(logits, hp, bias=None):
    l64 = f64(logits)
    idx, w = run(logits, hp, bias)
    want_idx, want = route(l64, None if bias is None else f64(bias), hp)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    got = f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.all(np.nan_to_num(np.abs(got - want)) <= np.nan_to_num(np.abs(want)) * (min(reach(l64), 110.0) + 64) * 2.0 ** -24 + 1e-37)
    return idx


def check_grad(logits, hp, idx, dw):
    l64, d64, at = f64(logits), f64(dw), idx.cpu().numpy()
    got, want = f64(run_grad(logits, hp, idx, dw)), None
    want = route_grad(l64, at, d64, hp)
    valid = (at >= 0) & (at < l64.shape[1])
    g = np.where(valid, np.abs(np.where(valid, d64, 0.0)) * abs(hp.scale), 0.0).max(1, keepdims=True)
    # two terms, each as far off as a weight, and the result's rounding
    tol = 2 * (min(reach(l64), 110.0) + 64) * 2.0 ** -24 * g + HALF_STEP[logits.dtype] * np.abs(want) * 1.001
    tol += 2.0 ** -25 if logits.dtype == torch.float16 else 1e-37  # half a step of the smallest numbers
    assert got.shape == want.shape and np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


def normal(seed, *shape, std=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * std


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (3, 2, 2), (70, 8, 2), (5, 31, 31), (33, 64, 6), (130, 65, 8), (9, 128, 1),
                                                 (300, 160, 6), (67, 256, 8), (20, 257, 16), (11, 512, 32), (6, 1000, 32), (4, 1024, 4)])
def test_sizes(dtype, score, tokens, experts, topk):
    logits = normal(tokens * experts, tokens, experts).to(DTYPES[dtype])
    for renormalise in (0, 1):
        hp = HP(topk, score, renormalise, scale=2.5)
        idx = check(logits, hp)
        check_grad(logits, hp, idx, normal(3, tokens, topk))
        check(logits, hp, normal(5, experts, std=0.1))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("experts,groups,top_groups,topk", [(8, 2, 1, 3), (8, 8, 3, 3), (64, 4, 2, 8), (160, 8, 3, 6), (256, 8, 4, 8),
                                                            (320, 64, 5, 16), (1000, 10, 2, 7), (60, 12, 12, 4), (96, 3, 2, 32)])
def test_groups(score, experts, groups, top_groups, topk):
    for seed, best, bias, dtype in ((1, 2, True, "f32"), (2, 1, True, "bf16"), (3, 1, False, "f32"), (4, 2, False, "f32")):
        logits = normal(seed * experts, 97, experts).to(DTYPES[dtype])
        hp = HP(topk, score, 1, groups, top_groups, best, 1.0)
        check(logits, hp, normal(9, experts, std=0.2) if bias else None)


@pytest.mark.parametrize("experts,topk", [(8, 3), (64, 8), (200, 8), (256, 16)])
def test_equal_logits_and_equal_choices(experts, topk):
    """Many equal values: the lower index first, in both the plain order and the
    one with a bias (equal logits and equal bias are equal choices)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    # -1, 0 and 2: two pairs have the same sum of scores only where they are the same
    logits = torch.randint(-1, 2, (50, experts), generator=g, device=DEV).float()
    logits[logits > 0] = 2.0
    logits[0] = 0.0
    bias = torch.randint(0, 2, (experts,), generator=g, device=DEV).float() * 0.5
    for score in (SOFT, SIG):
        check(logits, HP(topk, score, 1))
        check(logits, HP(topk, score, 0), bias)
        check(logits, HP(min(topk, experts // 4 * 2), score, 0, 4, 2, 1), bias)
        check(logits, HP(min(topk, experts // 4 * 2), score, 0, 4, 2, 2))
        check(logits, HP(min(topk, experts // 4 * 2), score, 0, 4, 2, 1))


@pytest.mark.parametrize("experts", [12, 64, 256, 700])
def test_choices_closer_than_fp32(experts):
    """Logits next to each other in fp32 around a bias that makes the choices
    differ by less than fp32 shows; and a bias far larger than the scores."""
    base = normal(8, 40, experts, std=0.5)
    near = torch.nextafter(base[:, :1].expand(-1, experts), torch.full((), 9.0, device=DEV)).contiguous()
    near[:, ::2] = base[:, :1]
    bias = torch.where(torch.arange(experts, device=DEV) % 3 == 0, 1e-7, 0.0)
    for score in (SOFT, SIG):
        check(near, HP(4, score, 1), bias)
        check(near, HP(4, score, 1))
        check(base, HP(4, score, 1), normal(10, experts, std=1e6))
        check(base, HP(4, score, 1), normal(11, experts, std=1e-9) + 1000.0)
        check(near, HP(4, score, 1, 4, 2, 2), bias)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renormalise", [0, 1])
def test_masks_and_values_out_of_range(dtype, score, renormalise):
    dt = DTYPES[dtype]
    logits = normal(20, 12, 96).to(dt)
    inf, low = math.inf, torch.finfo(dt).min
    logits[0] = -inf                      # nothing is open
    logits[1, 3:] = -inf                  # fewer than topk are
    logits[2, ::2] = -inf
    logits[3] = low                       # masked by the lowest value
    logits[4, 5:90] = low
    logits[5, 7] = inf                    # counts as the largest float
    logits[6, 7] = logits[6, 50] = inf
    logits[7, 11] = math.nan              # the row's weights are NaN
    logits[8, 0:96:3] = math.nan
    logits[8, 1:96:3] = -inf
    logits[9] = torch.finfo(dt).max
    logits[10] = -200.0                   # scores below fp32's range
    logits[11] = 200.0
    bias = normal(21, 96, std=0.1)
    bias[40] = -inf
    bias[41] = math.nan
    bias[42] = inf
    for hp in (HP(5, score, renormalise), HP(5, score, renormalise, 8, 2, 2), HP(5, score, renormalise, 8, 2, 1)):
        for b in (None, bias):
            idx = check(logits, hp, b)
            keep = torch.tensor([0, 1, 2, 3, 4, 9, 10, 11], device=DEV)
            dw = normal(22, 12, 5)
            dw[idx < 0] = math.nan        # beside no expert: not looked at
            check_grad(logits[keep].contiguous(), hp, idx[keep].contiguous(), dw[keep].contiguous())


def test_the_largest_floats_gradient_is_finite():
    logits = normal(30, 2, 16)
    logits[0, 3] = math.inf
    hp = HP(4, SOFT, 0)
    idx = check(logits, hp)
    d = run_grad(logits, hp, idx, normal(31, 2, 4))
    assert torch.isfinite(d).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_that_lie_apart(dtype):
    """Rows at a distance that begin at any element give the bits of dense ones,
    and nothing between the gradient's rows changes."""
    dense = normal(40, 21, 100).to(DTYPES[dtype])
    loose = spread(dense, 5)
    dw = normal(41, 21, 6)
    for hp in (HP(6, SOFT, 0), HP(6, SIG, 1, 4, 2, 2)):
        a, b = run(dense, hp), run(loose, hp)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        whole, view = apart(21, 100, dense.dtype, 3, fill=77.0)
        osa.optim_route_grad(loose, hp, a[0], dw, view)
        assert torch.equal(view, run_grad(dense, hp, a[0], dw))
        assert float(whole[0]) == 77.0 and bool((whole[1:].view(21, 103)[:, 100:] == 77.0).all())


def test_the_same_expert_twice_and_indices_out_of_range():
    logits = normal(50, 6, 40)
    idx = torch.randint(0, 40, (6, 7), device=DEV, dtype=torch.int32)
    idx[0] = 5
    idx[1, 2:5] = idx[1, 0]
    idx[2] = torch.tensor([40, 41, -1, -2 ** 31, 2 ** 31 - 1, 0, 39], dtype=torch.int32)
    idx[3] = -1
    for score in (SOFT, SIG):
        for renormalise in (0, 1):
            check_grad(logits, HP(7, score, renormalise, scale=0.5), idx, normal(51, 6, 7))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renormalise", [0, 1])
def test_gradient_against_differences(score, renormalise):
    """Central differences, in 64 bits, of the weights' product with dweights: a
    step of 1e-4 leaves an error of a third derivative's size, below 1e-7."""
    hp = HP(5, score, renormalise, scale=1.5)
    logits, dw = normal(60, 7, 23), normal(61, 7, 5)
    idx, _ = run(logits, hp)
    got, l64, d64, at = f64(run_grad(logits, hp, idx, dw)), f64(logits), f64(dw), idx.cpu().numpy()
    h = 1e-4
    for t in range(7):
        for e in range(23):
            up, down = l64[t].copy(), l64[t].copy()
            up[e] += h
            down[e] -= h
            slope = ((weights_of(up, at[t], hp) - weights_of(down, at[t], hp)) * d64[t]).sum() / (2 * h)
            assert abs(got[t, e] - slope) <= 2e-6 * (1 + np.abs(d64[t]).max() * 1.5)


def test_no_tokens_and_a_scale_of_nothing():
    osa.optim_route(torch.empty(0, 8, device=DEV), HP(2), torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV))
    logits = normal(70, 3, 8)
    idx, w = run(logits, HP(2, scale=0.0))
    assert float(w.abs().max()) == 0.0 and torch.equal(idx, run(logits, HP(2))[0])
    assert float(run_grad(logits, HP(2, scale=0.0), idx, normal(71, 3, 2)).abs().max()) == 0.0


def test_large_batch_repeats_and_agrees_with_small_ones():
    """Every token of a large batch has the result it has alone."""
    logits = normal(80, 40000, 256)
    bias = normal(81, 256, std=0.05)
    hp = HP(8, SIG, 1, 8, 4, 2, 2.5)
    idx, w = run(logits, hp, bias)
    again = run(logits, hp, bias)
    assert torch.equal(idx, again[0]) and torch.equal(w, again[1])
    for t in (0, 1, 1023, 20000, 39999):
        one = run(logits[t:t + 1].contiguous(), hp, bias)
        assert torch.equal(one[0][0], idx[t]) and torch.equal(one[1][0], w[t])
    some = torch.arange(0, 40000, 400, device=DEV)
    check(logits[some].contiguous(), hp, bias)


@pytest.mark.parametrize("experts", [16, 256])
def test_the_balance_bias(experts):
    loads = torch.randint(0, 50, (experts,), device=DEV)
    loads[3] = int(loads.sum() - loads[3]) // (experts - 1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), loads.cumsum(0)]).to(torch.int32)
    bias, rate, found = normal(90, experts), torch.tensor([1e-3], device=DEV), torch.zeros(1, device=DEV)
    before = bias.clone()
    osa.optim_step_route_bias(offsets, bias, rate, found_inf=found)
    n = loads.tolist()
    sign = torch.tensor([float(np.sign(sum(n) - x * experts)) for x in n], device=DEV)
    assert torch.equal(bias, before + rate * sign)
    found.fill_(1.0)
    osa.optim_step_route_bias(offsets, bias, rate, found_inf=found)
    assert torch.equal(bias, before + rate * sign)
    far = torch.tensor([0] + [2 ** 31 - 1] * 2, dtype=torch.int32, device=DEV)  # loads past 2^31 / experts
    b2 = torch.zeros(2, device=DEV)
    osa.optim_step_route_bias(far, b2, rate)
    assert b2.tolist() == [-rate.item(), rate.item()]
