"""Checks of include/optim_muon.h that need no GPU: exports, plan sizing,
refusals of lists and of hyperparameters.  Device pointers are fake integers,
never read."""
import math
import os
import re

import pytest

import optimizer_step_adamw_amd as osa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(osa.LIB_PATH):
        osa.build_library()
    return osa.lib()


def refused(code, fn):
    with pytest.raises(osa.OptimError) as ei:
        fn()
    assert ei.value.code == code and len(str(ei.value)) > 20, str(ei.value)


def matrices(shapes, **kw):
    n = len(shapes)
    at = lambda j: [A + (4 * k + j << 36) for k in range(n)]  # noqa: E731
    args = dict(params=at(0), grads=at(1), m=at(2), weight_decay=[0.0] * n, numel=[k * r * c for k, r, c in shapes],
                rows=[r for _, r, _ in shapes], cols=[c for _, _, c in shapes])
    args.update(kw)
    return osa.TensorList(**args)


def size(tl, opts=None):
    return osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_MUON, opts)


def test_exports(L):
    text = open(os.path.join(ROOT, "include", "optim_muon.h")).read()
    declared = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(optim_\w+)\s*\(", text, re.M))
    assert declared == set(osa.EXPORTED_MUON)
    for name in declared:
        assert hasattr(L, name), name


def test_workspace(L):
    one = size(matrices([(1, 100, 60)]))
    assert 0 < one < size(matrices([(4, 100, 60)])) < size(matrices([(4, 1000, 600)]))
    # a bound on a run's workspace: one matrix at a time
    assert size(matrices([(64, 512, 512)]), osa.optim_plan_opts(segment_bytes=1)) < size(matrices([(64, 512, 512)])) / 8
    assert size(matrices([])) > 0 and size(matrices([(0, 5, 7)])) > 0 and size(matrices([(1, 1, 1)])) > 0


def test_lists_that_do_not(L):
    ok = [(2, 30, 20)]
    assert size(matrices(ok)) > 0
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, rows=[0])))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, cols=[-3])))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, rows=[(1 << 20) + 1])))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, rows=[7])))  # does not divide
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, rows=None)))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, cols=None)))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, m=None)))
    refused(osa.OPTIM_EINVAL, lambda: size(matrices(ok, m=[A])))  # the momentum is the parameter
    refused(osa.OPTIM_EALIGN, lambda: size(matrices(ok, grads=[A * 3 + 2])))
    refused(osa.OPTIM_EDTYPE, lambda: size(matrices(ok, grad_dtype=osa.OPTIM_F16)))
    refused(osa.OPTIM_EUNSUPPORTED, lambda: size(matrices(ok, param_dtype=osa.OPTIM_BF16)))  # no remainder
    refused(osa.OPTIM_EUNSUPPORTED, lambda: size(matrices([(1 << 27, 1, 1)])))  # too many matrices
    for opts in (osa.optim_plan_opts(grid=8), osa.optim_plan_opts(state_dtype=osa.OPTIM_BF16),
                 osa.optim_plan_opts(state_layout=osa.OPTIM_LAYOUT_INTERLEAVED)):
        refused(osa.OPTIM_EUNSUPPORTED, lambda: size(matrices(ok), opts))


def test_calls_without_a_plan(L):
    import ctypes
    hp = osa.optim_muon_hp()
    assert L.optim_step_muon(None, ctypes.byref(hp), A, None, None, A, None) == osa.OPTIM_EINVAL


def test_hyperparameter_struct_matches_the_header(L):
    """Five doubles and three 32-bit integers, padded to a double."""
    import ctypes
    assert ctypes.sizeof(osa.optim_muon_hp) == 56
    hp = osa.optim_muon_hp()
    assert (hp.momentum, hp.eps, hp.a, hp.b, hp.c, hp.steps, hp.nesterov) == (0.95, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1)
