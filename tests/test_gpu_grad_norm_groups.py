"""The rounding of gradient norms (optim_grad_norms) where it is largest.  A
16-byte group is a chain of fp32 additions: after a 1, 2^-24 is half a step and
is lost (to even), 7 times in a group of 8 and 3 times in one of 4.  The sum is
then off by 7 (3) * 2^-24 of itself, which is its bound; a norm of squares by half
of that.  The rounding to fp32 adds 2^-24."""
import math

import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [1, 500, 100_000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["l1", "l2"])
def test_every_addition_is_lost(kind, dtype, groups):
    n = 4 if dtype == torch.float32 else 8
    small = 2.0 ** (-24 if kind == "l1" else -12)
    if dtype == torch.float16 and kind == "l1":
        small = 2.0 ** -23  # scaled: 2^-24 is a subnormal number there
    first = small * 2.0 ** 24 if kind == "l1" else 1.0
    g = torch.full((groups, n), small, device=DEV)
    g[:, 0] = first
    g = g.to(dtype).reshape(-1)
    assert g.data_ptr() % 16 == 0
    plan = osa.Plan(osa.grad_list([g]), osa.OPTIM_ALGO_GRADS)
    total = torch.zeros(1, device=DEV)
    osa.optim_grad_norms(plan.handle, {"l1": osa.OPTIM_NORM_L1, "l2": osa.OPTIM_NORM_L2}[kind], None, 0.0, None, None, total, None)
    x = g.double().abs()
    want = float(x.sum()) if kind == "l1" else math.sqrt(float(x.square().sum()))
    room = (n - 1) * 2.0 ** -24 * (1.0 if kind == "l1" else 0.5) + 2.0 ** -24
    off = abs(total.item() - want) / want
    assert off <= room, (off, room)
