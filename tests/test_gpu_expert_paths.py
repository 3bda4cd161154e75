"""Experts' weight gradients by wide tiles, which take enough tiles to fill the
GPU, and two calls at once.  Against float64 with the tolerance of
test_gpu_expert_grad.py: the order of a run's additions is not part of it."""
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, say
from test_gpu_expert_grad import check, make

pytestmark = pytest.mark.gpu

# 20 experts of 3 x 5 wide tiles, sides off a tile by 8 and more; runs of 0, 1, below, at and above whole steps
RUNS = [0, 1, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 0, 200, 255, 256, 257, 300, 7, 0]
SIZES = [(520, 1032), (768, 1280), (1272, 640)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", SIZES)
def test_wide_tiles(m, n, dtype, out, accumulate):
    say(m, n, dtype, out, accumulate)
    scale = torch.tensor([0.5], device=DEV)
    for kw in ({}, dict(before=3, behind=5), dict(padx=8, pady=24)):
        x, y, o, dw, off = make(RUNS, m, n, dtype, out, **kw)
        old = dw.clone()
        osa.optim_expert_grad(x, y, o, dw, accumulate=accumulate, scale=scale)
        check(x, y, off, old, dw, accumulate, 0.5)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 9), (7, 300), (130, 129), (257, 15)])
def test_odd_columns_and_ends_of_runs(m, n, out):
    """Whole steps of odd matrices read ahead by up to 8 rows: runs that end on both sides of that, the last at the end
    of the array, and columns, rows between and rows outside that hold NaN."""
    runs = [71, 72, 73, 0, 135, 136, 137, 64, 8, 199, 200, 201, 72]
    for kw in ({}, dict(before=1, behind=1), dict(padx=1, pady=5, shift=1), dict(padx=7)):
        x, y, o, dw, off = make(runs, m, n, torch.bfloat16, out, seed=9, **kw)
        old = dw.clone()
        osa.optim_expert_grad(x, y, o, dw, accumulate=True)
        check(x, y, off, old, dw, True, 1.0)


def test_two_calls_at_once():
    cases = [make(RUNS, m, n, torch.bfloat16, torch.float32, seed=5) for m, n in SIZES[:2]]
    want = []
    for x, y, o, dw, _ in cases:
        ref = torch.empty_like(dw)
        osa.optim_expert_grad(x, y, o, ref)
        want.append(ref)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for (x, y, o, dw, _), s in zip(cases, streams):
            dw.fill_(float("nan"))
        torch.cuda.synchronize()
        for (x, y, o, dw, _), s in zip(cases, streams):
            osa.optim_expert_grad(x, y, o, dw, stream=s)
        torch.cuda.synchronize()
        for (_, _, _, dw, _), ref in zip(cases, want):
            assert torch.equal(dw, ref)
