"""The operators on gradients and the steps together, as a training loop of a
mixture of experts uses them: weight gradients accumulate over two
micro-batches of routed rows into the arrays that the plans hold; norms over
the matrices' list and the vectors' list make one norm; both are clipped in
place by it; Muon steps the experts' and the router's matrices, AdamW the
vectors.  Three iterations, the second with an overflow (skipped), against
the same loop in float64.

The float64 loop takes each iteration's parameters and states as they are on
the GPU, so tolerances are one iteration's: expert gradients to 2e-6 of their
norm (sums of at most 130 terms in fp32, 130 * 2^-24, beside two roundings),
Muon's direction to 2.1e-4 as in its own tests plus the gradients' error times
the polynomial's largest growth, 3.44^5 = 485, AdamW's step to 2e-6."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
import oracle
from gpu_support import DEV, DevScalars, all_equal
from test_gpu_muon import direction64

pytestmark = pytest.mark.gpu

E, D, F, T = 6, 72, 136, 260
LOSS_SCALE = 1024.0
MAX_NORM = 0.5


def routed(gen):
    """Rows sorted by expert, one expert without any, bounds on the device."""
    which = torch.randint(0, E - 1, (T,), generator=gen, device=DEV)
    which = torch.where(which >= 3, which + 1, which)  # expert 3 gets none
    counts = torch.bincount(which, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = counts.cumsum(0).to(torch.int32)
    x = torch.randn(T, D, generator=gen, device=DEV).to(torch.bfloat16)
    dy = (torch.randn(T, F, generator=gen, device=DEV) * 1e-2 * LOSS_SCALE).to(torch.bfloat16)
    return x, dy, off


def test_a_training_loop_of_experts():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(101)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device=DEV) * std  # noqa: E731
    w, router = rnd(E, D, F, std=0.02), rnd(E, D, std=0.02)
    bias, scale = rnd(E * F, std=0.02), rnd(D, std=0.02)
    mats, vecs = [w, router], [bias, scale]
    gm, gv = [torch.zeros_like(p) for p in mats], [torch.zeros_like(p) for p in vecs]
    mm, mv, vv = ([torch.zeros_like(p) for p in q] for q in (mats, vecs, vecs))
    muon = osa.Plan(osa.TensorList(mats, gm, m=mm, weight_decay=[0.1, 0.1], rows=[D, E], cols=[F, D]), osa.OPTIM_ALGO_MUON)
    adam = osa.Plan(osa.TensorList(vecs, gv, m=mv, v=vv, weight_decay=[0.0, 0.0]), osa.OPTIM_ALGO_ADAMW)
    lists = [osa.Plan(osa.grad_list(g), osa.OPTIM_ALGO_GRADS) for g in (gm, gv)]
    sc, sca = DevScalars(0.02, inv_scale=1 / LOSS_SCALE), DevScalars(1e-3)
    totals, total, coef = torch.zeros(2, device=DEV), torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    hp, ahp = osa.optim_muon_hp(), osa.optim_adamw_hp(0.9, 0.999, 1e-8)
    applied = 0
    for it in range(3):
        batches = [routed(gen) for _ in range(2)]
        others = [rnd(E, D, std=1e-2 * LOSS_SCALE), rnd(E * F, std=1e-2 * LOSS_SCALE), rnd(D, std=1e-2 * LOSS_SCALE)]
        if it == 1:
            others[1][77] = math.inf
        before = [p.clone() for p in mats + vecs + mm + mv + vv]
        # gradients
        for k, (x, dy, off) in enumerate(batches):
            osa.optim_expert_grad(x, dy, off, gm[0], accumulate=k > 0)
        for g, o in zip([gm[1]] + gv, others):
            g.copy_(o)
        gw64 = np.zeros((E, D, F))
        for x, dy, off in batches:
            o = off.tolist()
            for e in range(E):
                gw64[e] += x[o[e]:o[e + 1]].double().cpu().numpy().T @ dy[o[e]:o[e + 1]].double().cpu().numpy()
        assert np.linalg.norm(gm[0].double().cpu().numpy() - gw64) <= 2e-6 * np.linalg.norm(gw64)
        assert float(gm[0][3].abs().max()) == 0.0
        # one norm, clipped by it
        sc.found_inf.zero_()
        for plan, g, t in zip(lists, (gm, gv), (totals[:1], totals[1:])):
            osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, sc.inv_scale, 0.0, sc.found_inf, None, t, None)
        osa.optim_clip_coef(totals, 2, osa.OPTIM_NORM_L2, sc.inv_scale, MAX_NORM, total, coef)
        for plan in lists:
            osa.optim_clip_grads(plan.handle, coef, sc.found_inf)
        g64 = [gw64] + [o.double().cpu().numpy() for o in others]
        n64 = math.sqrt(sum(float((g ** 2).sum()) for g in g64)) / LOSS_SCALE
        # both steps, unscaled by the clip
        osa.optim_step_muon(muon.handle, hp, sc.lr, None, sc.found_inf, sc.step)
        osa.optim_step_adamw(adam.handle, ahp, sca.lr, None, sc.found_inf, sca.step)
        torch.cuda.synchronize()
        now = mats + vecs + mm + mv + vv
        if it == 1:
            assert sc.found_inf.item() == 1.0 and all_equal(before, now) and sc.step.item() == sca.step.item() == applied
            continue
        applied += 1
        assert sc.found_inf.item() == 0.0 and sc.step.item() == sca.step.item() == applied
        assert abs(total.item() - n64) <= 2e-6 * n64 and n64 > MAX_NORM
        c64 = MAX_NORM / (n64 + 1e-6) / LOSS_SCALE
        p0 = [b.double().cpu().numpy() for b in before]
        for i, (p, shape) in enumerate(zip(mats, ((E, D, F), (1, E, D)))):
            g = g64[i] * c64
            m = 0.95 * p0[4 + i] + g
            o = direction64((0.95 * m + g).reshape(shape))
            f = 0.2 * math.sqrt(max(shape[1:])) * float(np.float32(0.02))
            want = p0[i].reshape(shape) * (1 - float(np.float32(0.02)) * 0.1) - f * o
            err = np.linalg.norm(p.double().cpu().numpy().reshape(shape) - want)
            assert err <= f * (2.1e-4 + 485 * 2e-6) * np.linalg.norm(o) + 2.0 ** -22 * np.linalg.norm(want), (it, i, err)
        for i, p in enumerate(vecs):
            q, m, v = p0[2 + i].copy(), p0[6 + i].copy(), p0[8 + i].copy()
            oracle.adamw_step(q, m, v, g64[2 + i] * c64, float(np.float32(1e-3)), 0.9, 0.999, 1e-8, 0.0, applied)
            got = p.double().cpu().numpy()
            assert np.max(np.abs(got - q) / np.maximum(np.abs(q), float(np.float32(1e-3)))) <= 2e-6, (it, i)
