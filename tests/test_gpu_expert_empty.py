"""Experts without rows (optim_expert_grad) get zeros, or keep their dW bit for
bit, whatever the scale is and in one piece as in several; the experts with rows
beside them are the product with that scale."""
import math

import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# the first: experts whose elements share a group of four; the others: whole groups
@pytest.mark.parametrize("m,n", [(3, 5), (64, 40), (130, 67), (136, 264)])
@pytest.mark.parametrize("scale", [math.inf, math.nan, -0.5])
@pytest.mark.parametrize("pieces", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_zeros_or_untouched(m, n, scale, pieces, accumulate, out):
    runs = [0, 9000, 0, 0, 3500, 0]
    off = [0]
    for r in runs:
        off.append(off[-1] + r)
    # rows of ones: every product is a whole number, exact in either order of summation
    x = torch.ones(off[-1], m, dtype=torch.bfloat16, device=DEV)
    y = torch.ones(off[-1], n, dtype=torch.bfloat16, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    dw = torch.zeros(len(runs), m, n, dtype=out, device=DEV)
    # what a sum with anything would change: -0 and a NaN with a payload
    bits(dw).fill_(-(2 ** 31) if out == torch.float32 else -(2 ** 15))
    bits(dw)[:, :, ::3] = 0x7F812345 if out == torch.float32 else 0x7F91
    old = dw.clone()
    ws = None
    if pieces:
        nbytes = osa.optim_expert_grad_workspace(len(runs), off[-1], m, n)
        assert nbytes > 0
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
    s = torch.tensor([scale], device=DEV)
    osa.optim_expert_grad(x, y, o, dw, accumulate=accumulate, scale=s, workspace=ws)
    for e, r in enumerate(runs):
        if r == 0:
            want = old[e] if accumulate else torch.zeros_like(old[e])
            assert torch.equal(bits(dw[e]), bits(want)) if accumulate else (dw[e] == 0).all(), e
        else:
            want = torch.full((m, n), float(r) * scale, device=DEV) + (old[e].float() if accumulate else 0.0)
            assert torch.equal(torch.nan_to_num(dw[e], nan=-1.0, posinf=1.0), torch.nan_to_num(want.to(out), nan=-1.0, posinf=1.0)), e
