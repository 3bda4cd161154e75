"""Dropout from a counter against its definition (the generator in Python's whole
numbers): which elements are dropped is exact; a kept one has a product and,
with a residual, a sum in fp32 and one rounding to its type."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, DTYPES, HALF_STEP, f64, kept

pytestmark = pytest.mark.gpu

HP = osa.optim_dropout_hp


def at_offset(n, dtype, by, seed):
    """n values that begin `by` elements into an allocation, with 99 around them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    whole = torch.full((n + by + 9,), 99.0, dtype=dtype, device=DEV)
    whole[by:by + n] = torch.randn(n, generator=g, device=DEV).to(dtype)
    return whole, whole[by:by + n]


def step_of(value):
    return torch.tensor([value], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n", [1, 7, 8, 9, 999, 4096, 20001])
@pytest.mark.parametrize("first,by", [(0, 0), (0, 1), (3, 0), (8, 3), (2 ** 35 - 5, 2)])
def test_against_the_definition(dtype, n, first, by):
    dt = DTYPES[dtype]
    for p, seed, step, site, with_residual in ((0.1, 2 ** 63 + 12345, 7, 0, False), (0.5, 3, 2 ** 31 - 1, 2 ** 32 - 1, True)):
        _, x = at_offset(n, dt, by, n)
        _, r = at_offset(n, dt, 2 * by, n + 1)
        whole, out = at_offset(n, dt, by + 1, n + 2)
        osa.optim_dropout(x, out, HP(p, seed, site, first), residual=r if with_residual else None, step=step_of(step))
        torch.cuda.synchronize()
        k = kept(n, p, seed, step, site, first)
        y = f64(x) * k
        want = y + f64(r) if with_residual else y
        # factor, product and sum in fp32, the result's rounding, fp16's smallest step
        tol = 3 * 2.0 ** -24 * (np.abs(y) + np.abs(want)) + HALF_STEP[dt] * np.abs(want) * 1.001 + (2.0 ** -25 if dtype == "f16" else 0)
        got = f64(out)
        assert np.all(np.abs(got - want) <= tol)
        if not with_residual:
            assert np.array_equal(got[k == 0], np.zeros((k == 0).sum()))
        assert bool((whole[:by + 1] == 99.0).all()) and bool((whole[by + 1 + n:] == 99.0).all())


def test_negative_steps_and_none():
    x = torch.randn(500, device=DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    osa.optim_dropout(x, a, HP(0.3, 11, 2))
    osa.optim_dropout(x, b, HP(0.3, 11, 2), step=step_of(0))
    assert torch.equal(a, b)
    osa.optim_dropout(x, a, HP(0.3, 11, 2), step=step_of(-1))
    assert np.array_equal(f64(a) == 0, kept(500, 0.3, 11, -1, 2, 0) == 0)


def test_pieces_have_the_mask_of_the_whole():
    x = torch.ones(10000, dtype=torch.bfloat16, device=DEV)
    whole = torch.empty_like(x)
    osa.optim_dropout(x, whole, HP(0.4, 77, 5, 13))
    for a, b in ((0, 1), (1, 9), (9, 4000), (4000, 4001), (4001, 10000)):
        part = torch.empty(b - a, dtype=torch.bfloat16, device=DEV)
        osa.optim_dropout(x[a:b], part, HP(0.4, 77, 5, 13 + a))
        assert torch.equal(part, whole[a:b])


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -16, 0.1, 0.5, 0.9, 0.99999, 1 - 2.0 ** -53])
def test_shares_and_means(p):
    """The share kept is that of the bar, within five deviations, and the mean stays."""
    n = 1 << 20
    out = torch.empty(n, device=DEV)
    osa.optim_dropout(torch.ones(n, device=DEV), out, HP(p, 5))
    keep = 1 - min(65535, math.floor(65536 * p + 0.5)) / 65536
    got = float((out != 0).double().mean())
    assert abs(got - keep) <= 5 * math.sqrt(keep * (1 - keep) / n)
    assert float(out.max()) == np.float32(1 / keep) if keep < 1 else bool((out == 1).all())


def test_dropped_elements_hide_what_they_hold():
    x = torch.full((4096,), math.nan, device=DEV)
    x[1::2] = math.inf
    out = torch.empty_like(x)
    osa.optim_dropout(x, out, HP(0.5, 9))
    gone = torch.from_numpy(kept(4096, 0.5, 9, 0, 0, 0) == 0).to(DEV)
    assert bool((out[gone] == 0).all()) and not torch.isfinite(out[~gone]).any()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_in_place_and_the_gradient(dtype):
    """In place on x or on the residual gives the same bits; the backward pass is
    the same call on the gradient, whose product with x is the forward's with dy."""
    dt = DTYPES[dtype]
    x, r = torch.randn(3001, device=DEV).to(dt), torch.randn(3001, device=DEV).to(dt)
    hp, out = HP(0.25, 21, 4), torch.empty(3001, dtype=dt, device=DEV)
    osa.optim_dropout(x, out, hp, residual=r, step=step_of(3))
    a, b = x.clone(), r.clone()
    osa.optim_dropout(a, a, hp, residual=r, step=step_of(3))
    osa.optim_dropout(x, b, hp, residual=b, step=step_of(3))
    assert torch.equal(a, out) and torch.equal(b, out)
    dx = torch.empty_like(x)
    osa.optim_dropout(torch.ones_like(x), dx, hp, step=step_of(3))
    assert np.array_equal(f64(dx) != 0, kept(3001, 0.25, 21, 3, 4, 0) != 0)


def test_no_elements():
    e = torch.empty(0, device=DEV)
    osa.optim_dropout(e, e, HP(0.5, 1))


def test_a_captured_step_draws_anew_at_every_replay():
    x, out, step = torch.randn(5000, device=DEV), torch.zeros(5000, device=DEV), step_of(0)
    hp = HP(0.5, 31, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            osa.optim_dropout(x, out, hp, step=step)
    torch.cuda.synchronize()
    seen = []
    for t in (1, 2, 3):
        step.fill_(t)
        g.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(x)
        osa.optim_dropout(x, want, hp, step=step)
        assert torch.equal(out, want)
        seen.append(want.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
