"""Tokens to the experts' rows and back, with their gradients, against the
definitions in 64 bits.  A sum over k choices in fp32 is off by (k + 2) 2^-24 of
the sum of its terms' magnitudes, dropout's factor and product and the residual
add three roundings, and the result has one to its type; a dot product over n
columns, summed in chains joined by halves, by less than n / 8 + 16 steps."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, DTYPES, HALF_STEP, apart, f64, kept, rows_of, spread

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1, 1), (1, 8, 256, 4096), (3, 2, 4, 7), (5, 3, 8, 8), (17, 8, 16, 100), (33, 4, 6, 1000), (9, 32, 40, 65), (64, 2, 8, 2049), (4, 5, 9, 8200)]
DROP = osa.optim_dropout_hp(0.3, 2 ** 40 + 3, 6)


def normal(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


class Layer:
    """Rows of `tokens` tokens: place, weights; some choices go nowhere, and a few
    rows belong to no choice."""

    def __init__(self, tokens, topk, experts, dim, dtype, seed=1, nowhere=0.2, more=3):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        idx = torch.rand(tokens, experts, generator=g, device=DEV).argsort(1)[:, :topk].to(torch.int32)
        idx[torch.rand(tokens, topk, generator=g, device=DEV) < nowhere] = -1
        off, place, _ = rows_of(idx.cpu().numpy(), experts)
        self.rows = int(off[-1]) + more
        self.place = torch.from_numpy(place).to(DEV)
        self.at = place
        self.weights = torch.rand(tokens, topk, generator=g, device=DEV)
        self.weights[self.place < 0] = math.nan  # beside no row: not looked at
        self.w = np.where(place >= 0, f64(self.weights), 0.0)
        self.x = normal(seed + 1, tokens, dim).to(dtype)
        self.y = normal(seed + 2, self.rows, dim).to(dtype)
        self.res = normal(seed + 3, tokens, dim).to(dtype)
        self.y[off[-1]:] = math.nan              # rows without a choice
        self.tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0

    def sums(self, w):
        """sum_j w y and the sum of its terms' magnitudes."""
        y = np.nan_to_num(f64(self.y))[self.at] * np.where(self.at >= 0, w, 0.0)[..., None]
        return y.sum(1), np.abs(y).sum(1)

    def factors(self, drop, step):
        t, d = self.x.shape
        return kept(t * d, drop.p, drop.seed, step, drop.site, drop.first).reshape(t, d) if drop else np.ones((t, d))


def step_of(value):
    return torch.tensor([value], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,dim", SIZES)
def test_gather(dtype, tokens, topk, experts, dim):
    s = Layer(tokens, topk, experts, dim, DTYPES[dtype])
    for weights in (None, s.weights):
        y = torch.full_like(s.y, 55.0)
        osa.optim_expert_gather(s.x, s.place, y, weights=weights)
        torch.cuda.synchronize()
        want = np.full(y.shape, 55.0)
        for t in range(tokens):
            for j in range(topk):
                if s.at[t, j] >= 0:
                    want[s.at[t, j]] = f64(s.x[t]) * (1.0 if weights is None else s.w[t, j])
        tol = 0.0 if weights is None else (2.0 ** -24 + HALF_STEP[s.x.dtype]) * np.abs(want) * 1.001 + s.tiny
        assert np.all(np.abs(f64(y) - want) <= tol)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,dim", SIZES)
@pytest.mark.parametrize("drop", [None, DROP])
def test_combine(dtype, tokens, topk, experts, dim, drop):
    s = Layer(tokens, topk, experts, dim, DTYPES[dtype])
    f = s.factors(drop, 12)
    for weights, residual in ((None, None), (s.weights, None), (s.weights, s.res), (None, s.res)):
        out = torch.full_like(s.x, 55.0)
        osa.optim_expert_combine(s.y, s.place, out, weights=weights, residual=residual, dropout=drop, step=step_of(12))
        torch.cuda.synchronize()
        total, terms = s.sums(np.ones_like(s.w) if weights is None else s.w)
        want = total * f + (0.0 if residual is None else f64(residual))
        tol = ((topk + 2) * terms * f + 3 * np.abs(total * f) + np.abs(want)) * 2.0 ** -24 + HALF_STEP[s.x.dtype] * np.abs(want) * 1.01 + s.tiny
        assert np.all(np.abs(f64(out) - want) <= tol)
        if residual is not None:  # in place
            again = residual.clone()
            osa.optim_expert_combine(s.y, s.place, again, weights=weights, residual=again, dropout=drop, step=step_of(12))
            assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,dim", SIZES)
@pytest.mark.parametrize("drop", [None, DROP])
def test_combine_grad(dtype, tokens, topk, experts, dim, drop):
    s = Layer(tokens, topk, experts, dim, DTYPES[dtype])
    d = f64(s.x) * s.factors(drop, 3)
    for weights in (None, s.weights):
        dy, dw = torch.full_like(s.y, 55.0), torch.full_like(s.weights, 55.0)
        osa.optim_expert_combine_grad(s.x, s.y, s.place, dy, weights=weights, dweights=dw, dropout=drop, step=step_of(3))
        torch.cuda.synchronize()
        want, got = np.full(dy.shape, 55.0), f64(dw)
        for t in range(tokens):
            for j in range(topk):
                r = s.at[t, j]
                if r < 0:
                    assert got[t, j] == 0.0
                    continue
                want[r] = d[t] * (1.0 if weights is None else s.w[t, j])
                terms = d[t] * f64(s.y[r])
                assert abs(got[t, j] - terms.sum()) <= (dim / 8 + 18) * 2.0 ** -24 * np.abs(terms).sum()
        assert np.all(np.abs(f64(dy) - want) <= (3 * 2.0 ** -24 + HALF_STEP[s.x.dtype]) * np.abs(want) * 1.01 + s.tiny)
        # one of the two alone, and dy where y lies
        only_dw, only_dy, inside, dw2 = torch.zeros_like(dw), torch.full_like(dy, 55.0), s.y.clone(), torch.zeros_like(dw)
        osa.optim_expert_combine_grad(s.x, s.y, s.place, None, weights=weights, dweights=only_dw, dropout=drop, step=step_of(3))
        osa.optim_expert_combine_grad(s.x, None, s.place, only_dy, weights=weights, dropout=drop, step=step_of(3))
        osa.optim_expert_combine_grad(s.x, inside, s.place, inside, weights=weights, dweights=dw2, dropout=drop, step=step_of(3))
        assert torch.equal(only_dw, dw) and torch.equal(only_dy, dy) and torch.equal(dw2, dw)
        used = torch.zeros(s.rows, dtype=torch.bool, device=DEV)
        used[s.place[s.place >= 0].long()] = True
        assert torch.equal(inside[used], dy[used]) and bool(torch.isnan(inside[~used]).all())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [40, 129])
def test_rows_that_lie_apart(dtype, dim):
    s = Layer(19, 3, 5, dim, DTYPES[dtype])
    x, y, res = spread(s.x, 3), spread(s.y, 5), spread(s.res, 1)
    a, (whole, b) = torch.zeros_like(s.x), apart(19, dim, s.x.dtype, 7, fill=77.0)
    osa.optim_expert_combine(s.y, s.place, a, weights=s.weights, residual=s.res, dropout=DROP)
    osa.optim_expert_combine(y, s.place, b, weights=s.weights, residual=res, dropout=DROP)
    assert torch.equal(a, b) and bool((whole[1:].view(19, dim + 7)[:, dim:] == 77.0).all()) and float(whole[0]) == 77.0
    for call in ("gather", "grad"):
        c, (whole, e) = torch.full_like(s.y, 77.0), apart(s.rows, dim, s.x.dtype, 9, fill=77.0)
        if call == "gather":
            osa.optim_expert_gather(s.x, s.place, c, weights=s.weights)
            osa.optim_expert_gather(x, s.place, e, weights=s.weights)
        else:
            dw = [torch.zeros_like(s.weights) for _ in range(2)]
            osa.optim_expert_combine_grad(s.x, s.y, s.place, c, weights=s.weights, dweights=dw[0], dropout=DROP)
            osa.optim_expert_combine_grad(x, y, s.place, e, weights=s.weights, dweights=dw[1], dropout=DROP)
            assert torch.equal(dw[0], dw[1])
        assert torch.equal(c, e) and bool((whole[1:].view(s.rows, dim + 9)[:, dim:] == 77.0).all())


def test_places_out_of_range_are_no_rows():
    s = Layer(6, 4, 8, 24, torch.float32, nowhere=0.0)
    bad = s.place.clone()
    bad[0] = torch.tensor([s.rows, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    none = bad.clone()
    none[0] = -1
    s.y = torch.nan_to_num(s.y)
    outs = []
    for p in (bad, none):
        out, y, dy, dw = torch.zeros_like(s.x), torch.zeros_like(s.y), torch.zeros_like(s.y), torch.ones_like(s.weights)
        osa.optim_expert_combine(s.y, p, out, weights=s.weights)
        osa.optim_expert_gather(s.x, p, y)
        osa.optim_expert_combine_grad(s.x, s.y, p, dy, weights=s.weights, dweights=dw)
        outs.append((out, y, dy, dw))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert float(outs[0][0][0].abs().max()) == 0.0 and float(outs[0][3][0].abs().max()) == 0.0


@pytest.mark.parametrize("tokens,rows,dim", [(0, 5, 8), (4, 0, 8), (4, 5, 0)])
def test_nothing_to_do(tokens, rows, dim):
    x, y = torch.ones(tokens, dim, device=DEV), torch.ones(rows, dim, device=DEV)
    place = torch.full((tokens, 2), -1, dtype=torch.int32, device=DEV)
    out, dw = torch.full_like(x, 3.0), torch.full((tokens, 2), 3.0, device=DEV)
    osa.optim_expert_gather(x, place, torch.ones_like(y))
    osa.optim_expert_combine(y, place, out)
    osa.optim_expert_combine_grad(x, y, place, torch.ones_like(y), dweights=dw)
    assert float(out.abs().sum()) == 0.0 and float(dw.abs().sum()) == 0.0


def test_the_gradient_of_a_gather():
    """Of a gather without weights: the sum over the rows.  With weights: the same
    with weights, and the dot products of x with the rows' gradients."""
    s = Layer(20, 4, 8, 72, torch.float32)
    dy = torch.nan_to_num(s.y)
    dx, dw = torch.zeros_like(s.x), torch.zeros_like(s.weights)
    osa.optim_expert_combine(dy, s.place, dx, weights=s.weights)
    osa.optim_expert_combine_grad(s.x, dy, s.place, None, dweights=dw)
    # y = w x is linear in either: <dy, y> = <dx, x> = <dw, w>
    y = torch.zeros_like(s.y)
    osa.optim_expert_gather(s.x, s.place, y, weights=s.weights)
    whole = (f64(dy) * f64(y)).sum()
    size = (np.abs(f64(dy)) * np.abs(f64(y))).sum()
    assert abs((f64(dx) * f64(s.x)).sum() - whole) <= 32 * 2.0 ** -24 * size
    assert abs((f64(dw) * s.w).sum() - whole) <= 32 * 2.0 ** -24 * size


def test_many_tokens_repeat_and_agree_with_few():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    t, k, d = 30000, 4, 520
    place = torch.randperm(t * k, generator=g, device=DEV).view(t, k).to(torch.int32)
    y, w = normal(4, t * k, d).to(torch.bfloat16), torch.rand(t, k, generator=g, device=DEV)
    x = normal(5, t, d).to(torch.bfloat16)
    out, dy, dw = torch.zeros_like(x), torch.zeros_like(y), torch.zeros_like(w)
    osa.optim_expert_combine(y, place, out, weights=w, dropout=DROP)
    osa.optim_expert_combine_grad(x, y, place, dy, weights=w, dweights=dw, dropout=DROP)
    again = torch.zeros_like(dw)
    osa.optim_expert_combine_grad(x, y, place, dy, weights=w, dweights=again, dropout=DROP)
    assert torch.equal(dw, again)
    for a in (0, 777, 29990):
        n, hp = 10, osa.optim_dropout_hp(DROP.p, DROP.seed, DROP.site, a * d)
        o, f, v = torch.zeros_like(x[:n]), torch.zeros_like(y), torch.zeros_like(w[:n])
        osa.optim_expert_combine(y, place[a:a + n], o, weights=w[a:a + n], dropout=hp)
        osa.optim_expert_combine_grad(x[a:a + n], y, place[a:a + n], f, weights=w[a:a + n], dweights=v, dropout=hp)
        at = place[a:a + n].flatten().long()
        assert torch.equal(o, out[a:a + n]) and torch.equal(v, dw[a:a + n]) and torch.equal(f[at], dy[at])
