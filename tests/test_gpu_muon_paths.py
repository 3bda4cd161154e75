"""The ways that the Muon step takes through larger lists: wide tiles with the
rest of a round by narrow ones, tiles shared by two groups of wavefronts, sums
in pieces, slabs joined four at a time, and the first size past the slabs.
Directions and parameters against float64 as in test_gpu_muon.py, with its
tolerance: none of these ways rounds more than the products counted there."""
import math

import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, DevScalars, all_equal, say
from test_gpu_muon import COEF, TOL_DIRECTION, State, step

pytestmark = pytest.mark.gpu

LISTS = {
    # over 256 wide tiles of X, tall and wide, sides off every tile; 384 + 30 of A
    "wide": [(60, 520, 600), (5, 700, 513), (1, 130, 300)],
    # ... and of A not half a round: the rest by narrow tiles
    "wide rest": [(31, 768, 768), (3, 515, 1025)],
    "pairs": [(2, 257, 300), (1, 300, 140)],
    "pieces": [(1, 1500, 140), (2, 401, 900), (1, 160, 160)],
    "pieces of both": [(1, 900, 1040), (1, 700, 650)],
    "slabs": [(1, 64, 5000), (3, 2100, 33), (1, 100, 2000), (2, 1300, 128), (1, 1, 20000)],
    "most slabs": [(1, 17, 32768), (1, 16384, 65), (1, 32769, 20), (1, 131072, 40)],
    # one slab too many for a matrix, and too many in all
    "past the slabs": [(1, 65537, 70), (1, 131073, 5)],
    "many slabs": [(97, 128, 1000), (2, 64, 700)],
}


def direction64(u, steps=5, eps=1e-7):
    x = u / (u.norm() + eps)
    for _ in range(steps):
        t = x.t().contiguous()
        a = x @ t if x.shape[0] <= x.shape[1] else t @ x
        b = COEF[1] * a + COEF[2] * (a @ a)
        x = COEF[0] * x + (b @ x if x.shape[0] <= x.shape[1] else x @ b)
    return x


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(LISTS))
def test_against_float64(name, kind):
    shapes = LISTS[name]
    st = State(shapes, seed=31, kind=kind, grad=torch.bfloat16 if kind == "bf16" else torch.float32)
    lr = float(np.float32(0.02))
    hp, sc = osa.optim_muon_hp(), DevScalars(lr)
    p0, m0 = [st.values(i).clone() for i in range(len(shapes))], [m.clone() for m in st.m]
    step(st, hp, sc)
    torch.cuda.synchronize()
    mu = float(np.float32(hp.momentum))
    for i, (k, r, c) in enumerate(shapes):
        g = st.g[i].float()
        m = m0[i] * mu
        m = m + g
        assert torch.equal(st.m[i], m), (name, shapes[i])
        u = m * mu
        u = (g + u).double().view(k, r, c)
        f = 0.2 * math.sqrt(max(r, c))
        assert hp.scale_kind == osa.OPTIM_MUON_SCALE_RMS and hp.nesterov == 1 and hp.steps == 5
        p64, got = p0[i].double().view(k, r, c), st.values(i).double().view(k, r, c)
        for q in range(k):
            o = direction64(u[q])
            err = float((got[q] - (p64[q] - lr * (0.1 * p64[q] + f * o))).norm())
            room = (TOL_DIRECTION + 2.0 ** -23) * lr * f * float(o.norm()) + 3 * 2.0 ** -24 * float(p64[q].norm())
            if q == 0:
                say(name, shapes[i], f"off {err:.3g} of {room:.3g}")
            assert err <= room, (name, shapes[i], q, err, room)
    assert sc.step.item() == 1


@pytest.mark.parametrize("name", list(LISTS))
def test_bits_do_not_depend_on_runs_or_streams(name):
    """Whole and in runs of little workspace; two plans at once on two streams."""
    ref = State(LISTS[name], seed=33)
    step(ref, osa.optim_muon_hp(), DevScalars(0.02))
    torch.cuda.synchronize()
    pair = [State(LISTS[name], seed=33, segment_bytes=cap) for cap in (1, 5_000_000)]
    streams, scalars = [torch.cuda.Stream() for _ in pair], [DevScalars(0.02) for _ in pair]
    torch.cuda.synchronize()
    for st, stream, sc in zip(pair, streams, scalars):
        step(st, osa.optim_muon_hp(), sc, stream=stream)
    torch.cuda.synchronize()
    for st in pair:
        assert all_equal(ref.buffers(), st.buffers()), name


@pytest.mark.parametrize("name", ["wide rest", "pieces of both", "slabs"])
def test_captured_and_replayed(name):
    st, twin = State(LISTS[name], seed=35), State(LISTS[name], seed=35)
    sc, tsc, hp = DevScalars(0.02), DevScalars(0.02), osa.optim_muon_hp()
    torch.cuda.synchronize()
    cs, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        with torch.cuda.graph(graph, stream=cs):
            step(st, hp, sc)
    torch.cuda.current_stream().wait_stream(cs)
    for k in range(4):
        for a, b in zip(st.g, twin.g):
            a.copy_(torch.randn_like(a) * 1e-3)
            b.copy_(a)
        graph.replay()
        step(twin, hp, tsc)
        torch.cuda.synchronize()
        assert all_equal(st.buffers(), twin.buffers()) and sc.step.item() == k + 1, k
