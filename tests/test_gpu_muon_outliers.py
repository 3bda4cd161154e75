"""The Muon step's direction (include/optim_muon.h) where elements of a matrix
differ by many orders of magnitude, against float64.

Tolerance, in the Frobenius norm: a factor of a product is held to 2^-22 of
itself and, where its low part is subnormal, to 2^-37 an element, so to 2^-22 of
its norm and 2^-37 sqrt(rows cols).  An iteration weighs its three products by
less than 10, each with two factors whose parts and sums are off by 3 times
that: 10 * 6 times.  Five iterations add up to less than 15 times one, by the
polynomial's slope (at most 3.9 on [0, 1.2]) and the growth of X itself:
900 (2^-22 |o| + 2^-37 sqrt(rows cols))."""
import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, DevScalars, say
from test_gpu_muon import State, direction64, step

pytestmark = pytest.mark.gpu

# one slab and several of each width, tiles, sums in pieces; tall and wide
SHAPES = [(64, 64), (100, 128), (40, 1000), (2000, 96), (256, 400), (400, 256), (140, 5000), (700, 600)]
SPREADS = {"one 1e3": 1e3, "one 1e6": 1e6, "one 1e9": 1e9, "one 1e30": 1e30, "rows 1e-6": 0.0, "columns 1e-12": 0.0}


@pytest.mark.parametrize("spread", list(SPREADS))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_elements_far_apart(rows, cols, spread):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(23)
    g = torch.randn(rows, cols, generator=gen, device=DEV)
    if spread.startswith("one"):
        g[rows // 2, cols // 3] = SPREADS[spread]
    elif spread.startswith("rows"):
        g[rows // 2:] *= 1e-6
    else:
        g[:, ::2] *= 1e-12
    st = State([(1, rows, cols)], p_std=0.0, wd=0.0)
    st.m[0].zero_()
    st.g[0].copy_(g.reshape(-1))
    hp = osa.optim_muon_hp(nesterov=0, scale_kind=osa.OPTIM_MUON_SCALE_NONE)
    step(st, hp, DevScalars(1.0))
    torch.cuda.synchronize()
    want = direction64(g.double().cpu().numpy()[None])[0]
    err = np.linalg.norm(-st.p[0].double().cpu().numpy().reshape(rows, cols) - want)
    # (and two roundings of the update, parameters of zero less lr 1 times it)
    room = (900 * 2.0 ** -22 + 2.0 ** -23) * np.linalg.norm(want) + 900 * 2.0 ** -37 * (rows * cols) ** 0.5
    say(rows, cols, spread, f"off {err:.3g} of {room:.3g}")
    assert err <= room, (err, room)
