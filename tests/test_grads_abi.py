"""Checks of include/optim_grads.h that need no GPU: exports, plan sizing and
refusals.  Device pointers are fake integers, never read: every call here is
refused, or sizes a plan."""
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


def grads(sizes, at=None, dtype=osa.OPTIM_F32, **kw):
    at = at or [A + (k << 24) for k in range(len(sizes))]
    return osa.TensorList([None] * len(sizes), at, weight_decay=[0.0] * len(sizes), numel=sizes, grad_dtype=dtype, **kw)


def size(tl, opts=None):
    return osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_GRADS, opts)


def test_exports(L):
    text = open(os.path.join(ROOT, "include", "optim_grads.h")).read()
    declared = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(optim_\w+)\s*\(", text, re.M))
    assert declared == set(osa.EXPORTED_GRADS)
    for name in declared:
        assert hasattr(L, name), name


@pytest.mark.parametrize("dtype", [osa.OPTIM_F32, osa.OPTIM_BF16, osa.OPTIM_F16])
def test_lists_that_plan(L, dtype):
    assert 0 < size(grads([4096], dtype=dtype)) < size(grads([4096] * 300, dtype=dtype))
    assert size(grads([])) > 0 and size(grads([0, 0])) > 0
    assert size(grads([1 << 40], [A])) > 0
    assert size(grads([5, 7], [A, A + 20], dtype=osa.OPTIM_F32)) > 0  # end to end in a bucket


def test_lists_that_do_not(L):
    refused(osa.OPTIM_EINVAL, lambda: size(grads([-1])))
    refused(osa.OPTIM_EINVAL, lambda: size(grads([(1 << 48) + 1])))
    refused(osa.OPTIM_EINVAL, lambda: size(grads([8], [0])))
    refused(osa.OPTIM_EALIGN, lambda: size(grads([8], [A + 2])))
    refused(osa.OPTIM_EALIGN, lambda: size(grads([8], [A + 1], dtype=osa.OPTIM_F16)))
    refused(osa.OPTIM_EDTYPE, lambda: size(grads([8], dtype=9)))
    # the same tensor twice, and two that share a byte
    refused(osa.OPTIM_EINVAL, lambda: size(grads([8, 8], [A, A])))
    refused(osa.OPTIM_EINVAL, lambda: size(grads([8, 8], [A, A + 28])))
    for opts in (osa.optim_plan_opts(grid=4), osa.optim_plan_opts(tile=2048), osa.optim_plan_opts(state_dtype=1),
                 osa.optim_plan_opts(state_layout=1)):
        refused(osa.OPTIM_EUNSUPPORTED, lambda: size(grads([8]), opts))


def test_calls_without_a_plan_or_with_bad_arguments(L):
    C, N = L.optim_grad_norms, L.optim_clip_coef
    assert C(None, 0, None, 1.0, None, None, A, None, None) == osa.OPTIM_EINVAL
    assert L.optim_clip_grads(None, A, None, None) == osa.OPTIM_EINVAL
    assert N(A, -1, 0, None, 1.0, A, A, None) == osa.OPTIM_EINVAL
    assert N(None, 2, 0, None, 1.0, A, A, None) == osa.OPTIM_EINVAL
    assert N(A, 2, 3, None, 1.0, A, A, None) == osa.OPTIM_EINVAL
    assert N(A, 2, -1, None, 1.0, A, A, None) == osa.OPTIM_EINVAL
    assert N(A, 2, 0, None, math.nan, A, A, None) == osa.OPTIM_EINVAL
    for bad in ((A + 2, 2, 0, None, 1.0, A, A), (A, 2, 0, A + 1, 1.0, A, A), (A, 2, 0, None, 1.0, A + 2, A),
                (A, 2, 0, None, 1.0, A, A + 3)):
        assert N(*bad, None) == osa.OPTIM_EALIGN


def test_binding_refuses_mixed_and_unknown_types(L):
    import torch
    with pytest.raises(ValueError):
        osa.grad_list([torch.zeros(3), torch.zeros(3, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        osa.grad_list([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError):
        osa.grad_list([torch.zeros(3)])  # not on a GPU


def test_expert_grad_refusals(L):
    import ctypes
    out = ctypes.c_size_t(0)
    W = L.optim_expert_grad_workspace
    assert W(4, 100, 64, 64, None) == osa.OPTIM_EINVAL
    for bad in ((-1, 10, 8, 8), (1, -1, 8, 8), (1, 10, -8, 8), (1, 10, 8, -8), (1, 1 << 31, 8, 8), (1, 10, 1 << 24, 8)):
        assert W(*bad, ctypes.byref(out)) == osa.OPTIM_EINVAL, bad
    assert W(1 << 20, 10, 1 << 20, 1 << 20, ctypes.byref(out)) == osa.OPTIM_EUNSUPPORTED
    assert W(64, 65536, 2048, 1024, ctypes.byref(out)) == osa.OPTIM_OK and out.value == 0
    assert W(1, 65536, 128, 128, ctypes.byref(out)) == osa.OPTIM_OK and out.value > 0
    assert W(0, 0, 0, 0, ctypes.byref(out)) == osa.OPTIM_OK and out.value == 0

    def call(x=A, ldx=64, dy=A + (1 << 30), ldy=32, dt=osa.OPTIM_BF16, off=A + (2 << 30), e=2, t=100, m=64, n=32,
             dw=A + (3 << 30), odt=osa.OPTIM_F32, scale=None, ws=None, nws=0):
        return L.optim_expert_grad(x, ldx, dy, ldy, dt, off, e, t, m, n, dw, odt, 0, scale, ws, nws, None)

    assert call(e=0) == call(m=0) == call(n=0, ldy=0) == osa.OPTIM_OK  # nothing to do, nothing launched
    for kw in (dict(ldx=63), dict(ldy=31), dict(x=None), dict(dy=None), dict(off=None), dict(dw=None), dict(e=-1), dict(t=-1),
               dict(dw=A + 64), dict(dw=A + (1 << 30)), dict(off=A + (3 << 30)), dict(ldx=1 << 24)):
        assert call(**kw) == osa.OPTIM_EINVAL, kw
    for kw in (dict(dt=osa.OPTIM_F32), dict(odt=osa.OPTIM_F16), dict(dt=5)):
        assert call(**kw) == osa.OPTIM_EDTYPE, kw
    for kw in (dict(x=A + 1), dict(dy=A + (1 << 30) + 1), dict(off=A + (2 << 30) + 2), dict(dw=A + (3 << 30) + 2), dict(scale=A + 3)):
        assert call(**kw) == osa.OPTIM_EALIGN, kw
    # a workspace that is too small or not aligned (the sizes want one)
    assert call(t=65536, e=1, ws=A + (4 << 30), nws=1000) == osa.OPTIM_EWORKSPACE
    assert call(t=65536, e=1, ws=A + (4 << 30) + 16, nws=1 << 30) == osa.OPTIM_EWORKSPACE
