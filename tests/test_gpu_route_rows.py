"""The experts' rows from the choices: whole numbers, equal to a plain sort, from
no token to many workgroups' worth, with choices that go nowhere."""
import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from route_support import DEV, rows_of

pytestmark = pytest.mark.gpu


def run(idx, experts, order=True):
    t, k = idx.shape
    n = osa.optim_route_rows_workspace(t, k, experts)
    ws = torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) if n else None
    off = torch.full((experts + 1,), -9, dtype=torch.int32, device=DEV)
    place = torch.full((t, k), -9, dtype=torch.int32, device=DEV)
    by = torch.full((t * k,), -9, dtype=torch.int32, device=DEV) if order else None
    osa.optim_route_rows(idx, off, place, order=by, workspace=ws)
    torch.cuda.synchronize()
    return off, place, by


def choices(seed, tokens, topk, experts, nowhere=0.0, skew=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.rand(tokens, topk, generator=g, device=DEV).pow(skew)
    idx = (x * experts).long().clamp(max=experts - 1).to(torch.int32)
    idx[torch.rand(tokens, topk, generator=g, device=DEV) < nowhere] = -1
    return idx


@pytest.mark.parametrize("tokens,topk,experts", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (7, 3, 5), (64, 1, 2), (65, 1, 1), (300, 2, 8),
                                                 (256, 8, 64), (257, 8, 64), (1000, 4, 1024), (3001, 5, 100), (2048, 1, 513)])
@pytest.mark.parametrize("nowhere", [0.0, 0.3, 1.0])
def test_small(tokens, topk, experts, nowhere):
    idx = choices(tokens + experts, tokens, topk, experts, nowhere, 2.0)
    off, place, order = run(idx, experts)
    want = rows_of(idx.cpu().numpy(), experts)
    for got, w in zip((off, place, order), want):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("tokens,topk,experts", [(4100, 1, 3), (65536, 8, 256), (70001, 7, 512), (30011, 6, 1000), (600001, 4, 16), (3000000, 2, 2), (6000001, 2, 300)])
@pytest.mark.parametrize("nowhere", [0.0, 0.1])
def test_large(tokens, topk, experts, nowhere):
    idx = choices(tokens, tokens, topk, experts, nowhere, 3.0)
    off, place, order = run(idx, experts)
    flat = idx.cpu().numpy().reshape(-1).astype(np.int64)
    by = np.where(flat < 0, experts, flat)
    want = np.argsort(by, kind="stable")
    counts = np.bincount(by, minlength=experts + 1)
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], counts.cumsum()[:-1]]))
    rows = counts[:experts].sum()
    got = order.cpu().numpy()
    assert np.array_equal(got[:rows], want[:rows]) and (got[rows:] == -1).all()
    at = np.empty(flat.size, np.int64)
    at[want] = np.arange(flat.size)
    assert np.array_equal(place.cpu().numpy().reshape(-1), np.where(flat < 0, -1, at))


def test_indices_out_of_range_and_no_order():
    idx = choices(5, 900, 4, 32)
    idx[3] = torch.tensor([32, 33, -5, 2 ** 31 - 1], dtype=torch.int32)
    idx[4, 0] = -2 ** 31
    plain = idx.clone()
    plain[(idx < 0) | (idx >= 32)] = -1
    a, b = run(idx, 32, order=False), run(plain, 32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_expert_takes_all_and_the_last_rows():
    idx = torch.full((20000, 2), 9, dtype=torch.int32, device=DEV)
    off, place, order = run(idx, 10)
    assert off.tolist() == [0] * 10 + [40000] and torch.equal(place.flatten(), torch.arange(40000, dtype=torch.int32, device=DEV))
    assert torch.equal(order, place.flatten())
