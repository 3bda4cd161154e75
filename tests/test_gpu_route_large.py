"""Sizes whose offsets pass 32 bits, and calls large enough to pass by the
caches: what lies far out equals the same call on that part alone, which the other
tests compare with the definitions."""
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV

pytestmark = pytest.mark.gpu

DROP = osa.optim_dropout_hp(0.25, 1234567, 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_of_more_than_2_31_elements(dtype, with_residual):
    n = (1 << 31) + 4099
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(1 << 20, generator=g, device=DEV).to(dtype).repeat(n // (1 << 20) + 1)[:n]
    out = torch.zeros_like(x)
    osa.optim_dropout(x, out, DROP, residual=x if with_residual else None)
    for a, b in ((0, 5000), ((1 << 31) - 2500, (1 << 31) + 2500), (n - 3000, n)):
        part = torch.zeros(b - a, dtype=dtype, device=DEV)
        hp = osa.optim_dropout_hp(DROP.p, DROP.seed, DROP.site, a)
        osa.optim_dropout(x[a:b], part, hp, residual=x[a:b] if with_residual else None)
        assert torch.equal(part, out[a:b])


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 70_000_001), (torch.float16, 150_000_003), (torch.float32, 40_000_001)])
def test_dropout_past_the_caches(dtype, n):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x, r = torch.randn(n, generator=g, device=DEV).to(dtype), torch.randn(n, generator=g, device=DEV).to(dtype)
    for residual in (None, r):
        out = torch.zeros_like(x)
        osa.optim_dropout(x, out, DROP, residual=residual)
        for a, b in ((0, 9000), (n // 2, n // 2 + 9001), (n - 8000, n)):
            part = torch.zeros(b - a, dtype=dtype, device=DEV)
            osa.optim_dropout(x[a:b].clone(), part, osa.optim_dropout_hp(DROP.p, DROP.seed, DROP.site, a),
                              residual=None if residual is None else residual[a:b].clone())
            assert torch.equal(part, out[a:b])
        again = x.clone()
        osa.optim_dropout(again, again, DROP, residual=residual)
        assert torch.equal(again, out)


@pytest.mark.parametrize("dtype,tokens,topk,dim", [(torch.bfloat16, 300_000, 2, 4096), (torch.float32, 40_000, 4, 4100)])
def test_rows_past_32_bits(dtype, tokens, topk, dim):
    """Rows of 2.5 to 5 GB, in an order that reaches all of them from the first tokens."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rows = tokens * topk
    place = (torch.arange(rows, device=DEV) * 7919 % rows).to(torch.int32).view(tokens, topk)
    w = torch.rand(tokens, topk, generator=g, device=DEV)
    base = torch.randn(1000, dim, generator=g, device=DEV).to(dtype)
    x = base.repeat(tokens // 1000, 1)
    y = torch.zeros(rows, dim, dtype=dtype, device=DEV)
    osa.optim_expert_gather(x, place, y, weights=w)
    some = torch.tensor([0, 1, tokens // 2, tokens - 1], device=DEV)
    at = place[some].long()
    assert torch.equal(y[at], (x[some].float()[:, None] * w[some][..., None]).to(dtype))
    out, dw = torch.zeros_like(x), torch.zeros_like(w)
    osa.optim_expert_combine(y, place, out, weights=w, residual=x, dropout=DROP)
    few = torch.zeros(4, dim, dtype=dtype, device=DEV)
    for i, t in enumerate(some.tolist()):
        hp = osa.optim_dropout_hp(DROP.p, DROP.seed, DROP.site, t * dim)
        osa.optim_expert_combine(y[at[i]].contiguous(), torch.arange(topk, dtype=torch.int32, device=DEV)[None], few[i:i + 1],
                                 weights=w[t:t + 1].contiguous(), residual=x[t:t + 1].contiguous(), dropout=hp)
    assert torch.equal(out[some], few)
    before = y[at].clone()
    osa.optim_expert_combine_grad(x, y, place, y, weights=w, dweights=dw, dropout=DROP)
    for i, t in enumerate(some.tolist()):
        hp, one = osa.optim_dropout_hp(DROP.p, DROP.seed, DROP.site, t * dim), torch.zeros(topk, dim, dtype=dtype, device=DEV)
        v = torch.zeros(1, topk, device=DEV)
        osa.optim_expert_combine_grad(x[t:t + 1].contiguous(), before[i].contiguous(), torch.arange(topk, dtype=torch.int32, device=DEV)[None],
                                      one, weights=w[t:t + 1].contiguous(), dweights=v, dropout=hp)
        assert torch.equal(y[at[i]], one) and torch.equal(dw[t:t + 1], v)


def test_logits_past_32_bits():
    tokens, experts, topk = 4_300_000, 256, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    logits = torch.randn(100_000, experts, generator=g, device=DEV).repeat(43, 1)
    logits[-1] = logits[-1].flip(0)
    hp = osa.optim_route_hp(topk, osa.OPTIM_ROUTE_SOFTMAX, 0)
    idx, w = torch.zeros(tokens, topk, dtype=torch.int32, device=DEV), torch.zeros(tokens, topk, device=DEV)
    osa.optim_route(logits, hp, idx, w)
    dl = torch.zeros_like(logits)
    osa.optim_route_grad(logits, hp, idx, w, dl)
    for a, b in ((0, 50), (2_100_000, 2_100_050), (tokens - 50, tokens)):
        i, v, d = idx[a:b].clone(), torch.zeros(b - a, topk, device=DEV), torch.zeros(b - a, experts, device=DEV)
        i.zero_()
        osa.optim_route(logits[a:b].clone(), hp, i, v)
        osa.optim_route_grad(logits[a:b].clone(), hp, i, v, d)
        assert torch.equal(i, idx[a:b]) and torch.equal(v, w[a:b]) and torch.equal(d, dl[a:b])


def test_more_tokens_than_a_launch():
    """2^25 tokens of 2 experts and some more: the last ones too."""
    tokens = (1 << 25) + 77
    logits = torch.zeros(tokens, 2, dtype=torch.bfloat16, device=DEV)
    logits[1::2, 1] = 1.0
    hp = osa.optim_route_hp(1)
    idx, w = torch.full((tokens, 1), 9, dtype=torch.int32, device=DEV), torch.zeros(tokens, 1, device=DEV)
    osa.optim_route(logits, hp, idx, w)
    want = torch.arange(tokens, device=DEV) % 2
    assert torch.equal(idx.flatten().long(), want) and bool((w == 1).all())
    dl, soft = torch.ones_like(logits), osa.optim_route_hp(1, osa.OPTIM_ROUTE_SOFTMAX, 0)
    osa.optim_route_grad(logits, soft, idx, w, dl)
    assert bool((dl[0::2] == torch.tensor([0.25, -0.25], device=DEV).bfloat16()).all())
    assert bool((dl[1::2] == dl[1]).all()) and float(dl[1, 1]) == -float(dl[1, 0]) != 0.0
