"""Sizes past what a launch can cover are refused when they are named, not when
they are launched (no GPU; device pointers are fake integers, never read)."""
import os

import pytest

import optimizer_step_adamw_amd as osa

A = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(osa.LIB_PATH):
        osa.build_library()


def refused(fn):
    with pytest.raises(osa.OptimError) as ei:
        fn()
    assert ei.value.code == osa.OPTIM_EUNSUPPORTED and len(str(ei.value)) > 20, str(ei.value)


def test_experts():
    """A block of 4 x 4 tiles of each: under 2^18 blocks."""
    assert osa.optim_expert_grad_workspace((1 << 18) - 1, 100, 1, 512) == 0
    assert osa.optim_expert_grad_workspace(63, 100, 1 << 15, 1 << 15) == 0
    for experts, m, n in ((1 << 18, 1, 512), (1 << 20, 1, 1), (1 << 17, 513, 1), (64, 1 << 15, 1 << 15), (2 ** 31 - 1, 1, 1)):
        refused(lambda: osa.optim_expert_grad_workspace(experts, 100, m, n))


def test_matrices():
    def size(count):
        tl = osa.TensorList([A], [2 * A], m=[3 * A], weight_decay=[0.0], numel=[4 * count], rows=[2], cols=[2])
        return osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_MUON)

    assert size(1000) > 0
    refused(lambda: size(1 << 23))


def test_gradients():
    def size(numel):
        tl = osa.TensorList([None], [A], weight_decay=[0.0], numel=[numel], grad_dtype=osa.OPTIM_BF16)
        return osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_GRADS)

    # items grow with the list: the table stays below 2^24 rows of 32 bytes
    for numel in (1 << 32, 1 << 40, 1 << 46):
        assert 0 < size(numel) < (1 << 24) * 64
