"""The gradient of routing where one expert has nearly all of the score: its own
element is the product of its score and a small difference, which is as exact
as the terms that make it up and no rounding of what is near one.

Element e is s_e (G_e (1 - s_e) - sum over the other choices of g_j s_j), G_e the
sum of g over the choices that name e (0: none).  In units of 2^-24 a score is off
by 2.3 |x| for its exponent (a difference and a product, each rounded once, and
the factor) and 2 for the exponential, the sum that divides it by as much and by
one for each of a lane's E / 16 terms and 8 for the joins, and 3 for the quotient:
R = 2.3 reach + E / 16 + 20 in all is above it.  Two such factors and four products
make an element, so it is off by 2 R + 8 of the sum of its terms' magnitudes, and
by its rounding to the logits' type."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, DTYPES, HALF_STEP, f64
from test_gpu_route import HP, SIG, SOFT, normal, run, run_grad

pytestmark = pytest.mark.gpu


def gradient(l, idx, dw, hp):
    """(gradient, sum of its terms' magnitudes) of a row, what is small summed by
    itself: 1 - s as the others' share."""
    at = [j for j in range(len(idx)) if 0 <= idx[j] < l.size and l[idx[j]] > -math.inf]
    out, size = np.zeros(l.size), np.zeros(l.size)
    if not at:
        return out, size
    g, e = hp.scale * dw[at], idx[at]
    if not hp.renormalise:
        x = np.exp(l - l.max())
        s = x / x.sum()
        for i in range(l.size):
            named = e == i
            rest = np.delete(x, i).sum() / x.sum()
            others = (g * s[e])[~named]
            out[i] = s[i] * (g[named].sum() * rest - others.sum())
            size[i] = s[i] * (np.abs(g[named]).sum() * rest + np.abs(others).sum())
        return out, size
    logs = l[e] if hp.score == SOFT else -np.logaddexp(0.0, -l[e])
    x = np.exp(logs - logs.max())
    w = x / x.sum()
    for i, to in enumerate(e):
        rest, others = np.delete(x, i).sum() / x.sum(), np.delete(g * w, i)
        by = w[i] * (1.0 if hp.score == SOFT else math.exp(-np.logaddexp(0.0, l[to])))
        out[to] += by * (g[i] * rest - others.sum())
        size[to] += by * (abs(g[i]) * rest + np.abs(others).sum())
    return out, size


def check(logits, hp, idx, dw):
    got, l64, d64, at = f64(run_grad(logits, hp, idx, dw)), f64(logits), f64(dw), idx.cpu().numpy()
    for t, l in enumerate(l64):
        fine = l[np.isfinite(l)]
        reach = float(fine.max() - fine.min())
        if hp.score == SIG:
            reach += 2 * float(np.abs(fine).max())  # (relative to the largest one, and by itself)
        want, size = gradient(l, at[t], d64[t], hp)
        tol = (2 * (2.3 * reach + l.size / 16 + 20) + 8) * 2.0 ** -24 * size + HALF_STEP[logits.dtype] * np.abs(want) * 1.001
        tol += 2.0 ** -25 if logits.dtype == torch.float16 else 1e-37
        assert np.all(np.abs(got[t] - want) <= tol), (t, np.max(np.abs(got[t] - want) / np.maximum(size, 1e-300)))


def rows(experts, dtype, topk, std=0.5):
    """Rows whose expert 5, 6, ... is 7 to 28 above the others, and its choices: that
    expert among them (first, last), named twice, and not at all."""
    logits = normal(experts, 12, experts, std=std)
    idx = torch.stack([torch.randperm(experts - 24, generator=torch.Generator().manual_seed(t))[:topk] + 24 for t in range(12)])
    for t in range(12):
        logits[t, 5 + t] += (7.0, 12.0, 17.0, 28.0)[t % 4]
        if t < 8:
            idx[t, 0 if t < 4 else topk - 1] = 5 + t
        if t in (2, 3) and topk > 1:
            idx[t, topk - 1] = 5 + t
        if t in (6, 7):
            idx[t, 0] = 5 + t
    logits[1, 30:] = -math.inf
    return logits.to(DTYPES[dtype]), idx.to(torch.int32).to(DEV), normal(7, 12, topk)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("experts", [48, 64, 200, 256, 512, 1000])
@pytest.mark.parametrize("topk", [1, 2, 8, 16, 20])
def test_of_the_whole_softmax(dtype, experts, topk):
    check_args = rows(experts, dtype, topk)
    check(check_args[0], HP(topk, SOFT, 0, scale=1.5), *check_args[1:])


def test_the_only_open_expert_has_none():
    logits = torch.full((9, 64), -math.inf, device=DEV)
    logits[:, 7] = normal(1, 9)
    for topk in (1, 8):
        hp = HP(topk, SOFT, 0)
        idx, _ = run(logits, hp)
        d = run_grad(logits, hp, idx, normal(2, 9, topk))
        assert float(d.abs().max()) == 0.0
