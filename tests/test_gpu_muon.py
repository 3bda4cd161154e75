"""The Muon step (include/optim_muon.h) against float64, element by element.

The momentum is fp32 without contraction and is checked bit for bit.  The
direction is compared in the Frobenius norm.  Its tolerance: every product of
an iteration is off by at most 3 * 2^-22 of its factors' norms (two factors
with 22 significant bits, the product of the low parts left out) and its fp32
sums by a like amount, and the polynomial's coefficients weigh the three
products of an iteration by less than 10: 10 * 6 * 2^-22 of X's norm per
iteration.  From one iteration to the next an error grows by the
polynomial's slope, at most 3.9 on [0, 1.2], while X's own norm grows by up to
3.44 until its singular values are near one, so five iterations add up to
less than 15 times one: 900 * 2^-22 = 2.1e-4.
The update is p - fma(lr wd, p, f x) in fp32: at most 2 roundings of the
parameter's scale and one of the update's."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, DevScalars, all_equal, say

pytestmark = pytest.mark.gpu

TOL_DIRECTION = 900 * 2.0 ** -22
COEF = (3.4445, -4.7750, 2.0315)
# sides of one, both sides of a tile and of a slab, tall and wide, stacks, odd columns
SHAPES = [(1, 1, 1), (1, 1, 7), (1, 5, 1), (2, 3, 5), (1, 64, 64), (1, 172, 64), (1, 64, 172), (1, 128, 128),
          (1, 129, 127), (1, 127, 129), (1, 130, 300), (1, 300, 131), (3, 40, 72), (2, 257, 33), (1, 1000, 408), (1, 96, 2000),
          (2, 64, 257), (1, 256, 64), (1, 65, 128), (2, 65, 130), (1, 1025, 17), (1, 1, 3000)]


def direction64(u, coef=COEF, steps=5, eps=1e-7):
    """Matrix by matrix in float64 on the CPU."""
    out = np.empty_like(u)
    for k in range(u.shape[0]):
        x = u[k] / (np.linalg.norm(u[k]) + eps) if np.linalg.norm(u[k]) + eps > 0 else u[k]
        for _ in range(steps):
            a = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
            b = coef[1] * a + coef[2] * a @ a
            x = coef[0] * x + (b @ x if x.shape[0] <= x.shape[1] else x @ b)
        out[k] = x
    return out


class State:
    """Parameters, gradients and momenta of a list of (count, rows, cols)."""

    def __init__(self, shapes, seed=1, grad=torch.float32, kind="f32", p_std=0.02, wd=0.1, shift=0, segment_bytes=0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)

        def normal(n, std):
            return torch.randn(n, generator=gen, device=DEV) * std

        def carve(n, dtype):  # `shift` elements behind a boundary
            return torch.empty(n + shift, dtype=dtype, device=DEV)[shift:]

        self.shapes, self.kind = shapes, kind
        ns = [k * r * c for k, r, c in shapes]
        self.master = [carve(n, torch.float32) for n in ns]
        self.m = [carve(n, torch.float32) for n in ns]
        self.g = [carve(n, grad) for n in ns]
        for x, m, g, n in zip(self.master, self.m, self.g, ns):
            x.copy_(normal(n, p_std))
            m.copy_(normal(n, 5e-3))
            g.copy_(normal(n, 1e-3))
        kw = {}
        if kind == "f32":
            self.p, code = self.master, osa.OPTIM_F32
        elif kind == "rem":
            self.p, self.r, code = [carve(n, torch.int16) for n in ns], [carve(n, torch.int16) for n in ns], osa.OPTIM_BF16
            for x, b, r in zip(self.master, self.p, self.r):
                osa.optim_remainder_split(x, b, r, x.numel())
            kw["remainders"] = self.r
        else:
            dt = torch.bfloat16 if kind == "bf16" else torch.float16
            self.p, code = [carve(n, dt) for n in ns], osa.OPTIM_BF16 if kind == "bf16" else osa.OPTIM_F16
            for x, b in zip(self.master, self.p):
                b.copy_(x)
            kw["master"] = self.master
        self.tl = osa.TensorList(self.p, self.g, m=self.m, weight_decay=[wd] * len(ns), rows=[r for _, r, _ in shapes],
                                 cols=[c for _, _, c in shapes], param_dtype=code,
                                 grad_dtype=osa.OPTIM_BF16 if grad == torch.bfloat16 else osa.OPTIM_F32, **kw)
        self.plan = osa.Plan(self.tl, osa.OPTIM_ALGO_MUON, segment_bytes=segment_bytes)

    def values(self, i):
        """fp32 parameter i."""
        if self.kind != "rem":
            return self.master[i]
        out = torch.empty(self.p[i].numel(), device=DEV)
        osa.optim_remainder_reconstruct(self.p[i], self.r[i], out, out.numel())
        return out

    def buffers(self):
        return list(self.p) + list(self.m) + ([] if self.kind == "f32" else self.r if self.kind == "rem" else self.master)


def step(st, hp, sc, stream=None):
    osa.optim_step_muon(st.plan.handle, hp, sc.lr, sc.inv_scale, sc.found_inf, sc.step, stream=stream)


def check_step(st, hp, sc, wd, lr, s):
    """One step on `st` against float64, from its state before."""
    p0 = [st.values(i).clone() for i in range(len(st.shapes))]
    m0 = [m.clone() for m in st.m]
    step(st, hp, sc)
    torch.cuda.synchronize()
    mu = float(np.float32(hp.momentum))
    for i, (k, r, c) in enumerate(st.shapes):
        g = st.g[i].float() * s
        m = m0[i] * mu
        m = m + g
        assert torch.equal(st.m[i], m), (i, st.shapes[i])
        u = m * mu
        u = g + u if hp.nesterov else m
        o = direction64(u.double().cpu().numpy().reshape(k, r, c), (hp.a, hp.b, hp.c), hp.steps, hp.eps)
        f = {osa.OPTIM_MUON_SCALE_NONE: 1.0, osa.OPTIM_MUON_SCALE_ASPECT: math.sqrt(max(1.0, r / c)),
             osa.OPTIM_MUON_SCALE_RMS: 0.2 * math.sqrt(max(r, c))}[hp.scale_kind]
        p64 = p0[i].double().cpu().numpy().reshape(k, r, c)
        want = p64 - lr * (wd * p64 + f * o)
        got = st.values(i).double().cpu().numpy().reshape(k, r, c)
        for q in range(k):
            err = np.linalg.norm(got[q] - want[q])
            room = (TOL_DIRECTION + 2.0 ** -23) * lr * f * np.linalg.norm(o[q]) + 3 * 2.0 ** -24 * np.linalg.norm(p64[q])
            say(st.shapes[i], q, f"off {err:.3g} of {room:.3g}")
            assert err <= room, (i, q, st.shapes[i], err, room)
        if st.kind in ("bf16", "f16"):
            assert torch.equal(st.p[i], st.master[i].to(st.p[i].dtype))


@pytest.mark.parametrize("nesterov", [0, 1])
def test_direction_alone(nesterov):
    """Parameters of zero, no decay, lr 1: the parameters are the direction."""
    st = State(SHAPES, seed=3, p_std=0.0, wd=0.0)
    hp = osa.optim_muon_hp(nesterov=nesterov, scale_kind=osa.OPTIM_MUON_SCALE_NONE)
    check_step(st, hp, DevScalars(1.0), 0.0, 1.0, 1.0)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["f32", "rem", "bf16", "f16"])
def test_three_steps(kind, grad, shift):
    st = State(SHAPES, seed=5, grad=grad, kind=kind, shift=shift)
    lr = float(np.float32(0.02))
    sc = DevScalars(lr, inv_scale=0.5)
    for t in range(3):
        hp = osa.optim_muon_hp(nesterov=t != 1, scale_kind=t)
        check_step(st, hp, sc, 0.1, lr, 0.5)
        for g in st.g:
            g.mul_(-0.7)
    assert sc.step.item() == 3


@pytest.mark.parametrize("coef,steps", [((1.5, -0.5, 0.0), 8), ((2.0, -1.5, 0.5), 1), ((3.4445, -4.7750, 2.0315), 2)])
def test_other_polynomials(coef, steps):
    st = State([(1, 70, 200), (1, 200, 70)], seed=7, p_std=0.0, wd=0.0)
    hp = osa.optim_muon_hp(a=coef[0], b=coef[1], c=coef[2], steps=steps, scale_kind=osa.OPTIM_MUON_SCALE_NONE)
    check_step(st, hp, DevScalars(1.0), 0.0, 1.0, 1.0)


@pytest.mark.parametrize("rank", [1, 3])
@pytest.mark.parametrize("value", [1.0, 1e-12, 1e15])
def test_few_strong_directions(rank, value):
    """Gradients of low rank, tiny or huge (eps 0)."""
    st = State([(1, 150, 260), (1, 260, 150)], seed=9, p_std=0.0, wd=0.0)
    for m, g, (k, r, c) in zip(st.m, st.g, st.shapes):
        m.zero_()
        g.copy_((torch.randn(r, rank, device=DEV) @ torch.randn(rank, c, device=DEV)).reshape(-1) * value)
    check_step(st, osa.optim_muon_hp(eps=0.0, scale_kind=osa.OPTIM_MUON_SCALE_NONE), DevScalars(1.0), 0.0, 1.0, 1.0)


@pytest.mark.parametrize("eps", [0.0, 1e-7])
def test_matrices_of_zeros_and_of_nan(eps):
    """A stack: zeros (update 0: decay alone), a NaN, an Inf, ordinary ones."""
    st = State([(5, 40, 72), (1, 100, 30)], seed=11)
    twin = State([(5, 40, 72), (1, 100, 30)], seed=11)
    n = 40 * 72
    for s in (st, twin):
        s.m[0][:n] = 0
        s.g[0][:n] = 0
    st.g[0][2 * n + 5], st.g[0][4 * n - 1] = math.nan, math.inf
    p0 = st.p[0][:n].clone()
    hp, sc, tsc = osa.optim_muon_hp(eps=eps), DevScalars(0.02), DevScalars(0.02)
    step(st, hp, sc)
    step(twin, hp, tsc)
    lw = float(np.float32(float(np.float32(0.02)) * 0.1))
    assert torch.allclose(st.p[0][:n].double(), p0.double() * (1 - lw), rtol=2.0 ** -23, atol=0)
    for q in (2, 3):
        assert torch.isnan(st.p[0][q * n:(q + 1) * n]).all()
    for q in (0, 1, 4):
        assert torch.equal(st.p[0][q * n:(q + 1) * n], twin.p[0][q * n:(q + 1) * n])
    assert torch.equal(st.p[1], twin.p[1])


def test_skip_schedule_and_counts():
    st = State(SHAPES[:8], seed=13)
    before = [b.clone() for b in st.buffers()]
    sc = DevScalars(0.02)
    osa.optim_plan_set_schedule(st.plan.handle, osa.OPTIM_SCHED_COSINE, 0.04, 0.0, 4, sc.iter)
    sc.found_inf.fill_(1.0)
    step(st, osa.optim_muon_hp(), sc)
    assert all_equal(before, st.buffers()) and sc.step.item() == 0 and sc.iter.item() == 1
    sc.found_inf.zero_()
    step(st, osa.optim_muon_hp(), sc)
    want = float(np.float32(0.04 * (1 + math.cos(math.pi / 4)) / 2))
    assert sc.step.item() == 1 and sc.iter.item() == 2 and sc.lr.item() == want
    assert not all_equal(before, st.buffers())


def test_empty_lists_still_count():
    for shapes in ([], [(0, 4, 4)]):
        st = State(shapes)
        sc = DevScalars(0.02)
        step(st, osa.optim_muon_hp(), sc)
        assert sc.step.item() == 1


def test_runs_streams_and_repeats_give_the_same_bits():
    ref = State(SHAPES, seed=15)
    step(ref, osa.optim_muon_hp(), DevScalars(0.02))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for cap in (0, 1, 3_000_000):
        st = State(SHAPES, seed=15, segment_bytes=cap)
        side.wait_stream(torch.cuda.current_stream())
        step(st, osa.optim_muon_hp(), DevScalars(0.02), stream=side)
        side.synchronize()
        assert all_equal(ref.buffers(), st.buffers()), cap


def test_check_and_norm_take_the_plan():
    st = State([(2, 100, 60), (1, 33, 33)], seed=17)
    fi, norm, clip = (torch.zeros(1, device=DEV) for _ in range(3))
    osa.optim_check_finite(st.plan.handle, fi)
    osa.optim_grad_norm(st.plan.handle, None, 1.0, fi, norm, clip)
    want = math.sqrt(sum(float(g.double().square().sum()) for g in st.g))
    assert fi.item() == 0 and abs(norm.item() - want) <= 1e-6 * want
    st.g[1][7] = math.inf
    osa.optim_check_finite(st.plan.handle, fi)
    assert fi.item() == 1


def test_captured_and_replayed():
    shapes = SHAPES[4:14]
    st, twin = State(shapes, seed=19), State(shapes, seed=19)
    sc, tsc, hp = DevScalars(0.02), DevScalars(0.02), osa.optim_muon_hp()
    torch.cuda.synchronize()
    cs, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        with torch.cuda.graph(graph, stream=cs):
            step(st, hp, sc)
    torch.cuda.current_stream().wait_stream(cs)
    for k in range(5):
        for a, b in zip(st.g, twin.g):
            a.copy_(torch.randn_like(a) * 1e-3)
            b.copy_(a)
        sc.found_inf.fill_(float(k == 2))
        tsc.found_inf.fill_(float(k == 2))
        graph.replay()
        step(twin, hp, tsc)
        torch.cuda.synchronize()
        assert all_equal(st.buffers(), twin.buffers()) and sc.step.item() == tsc.step.item() == (k + 1 if k < 2 else k), k


def test_refused_hyperparameters():
    st = State([(1, 8, 8)])
    sc = DevScalars(0.02)
    before = [b.clone() for b in st.buffers()]
    bad = [dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=math.nan), dict(eps=-1.0), dict(eps=math.inf),
           dict(a=math.nan), dict(steps=0), dict(steps=17), dict(scale_kind=3), dict(scale_kind=-1),
           dict(a=16.0), dict(a=4.0, b=0.0, c=0.0, steps=3), dict(b=-20.0, c=0.0), dict(c=50.0)]
    for kw in bad:
        with pytest.raises(osa.OptimError) as ei:
            step(st, osa.optim_muon_hp(**kw), sc)
        assert ei.value.code == osa.OPTIM_EINVAL, kw
    for args in ((None, sc.step), (sc.lr, None)):
        with pytest.raises(osa.OptimError):
            osa.optim_step_muon(st.plan.handle, osa.optim_muon_hp(), args[0], None, None, args[1])
    with pytest.raises(osa.OptimError):  # a plan of another algorithm
        osa.optim_step_lion(st.plan.handle, osa.optim_lion_hp(0.9, 0.99), sc.lr, None, None, sc.step)
    torch.cuda.synchronize()
    assert all_equal(before, st.buffers()) and sc.step.item() == 0
