"""An entry point that runs out of host memory returns a status with a message,
as every other failure does; it does not end the process.  Each call runs in a
process of its own whose address space is bounded once the library is loaded (no
GPU; device pointers are fake integers, never read)."""
import os
import subprocess
import sys

import pytest

import optimizer_step_adamw_amd as osa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import resource, sys
import optimizer_step_adamw_amd as osa
A = 1 << 40

def muon(count):
    tl = osa.TensorList([A], [2 * A], m=[3 * A], weight_decay=[0.0], numel=[4 * count], rows=[2], cols=[2])
    return lambda: osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_MUON)

def grads(numel):
    tl = osa.TensorList([None], [A], weight_decay=[0.0], numel=[numel], grad_dtype=osa.OPTIM_BF16)
    return lambda: osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_GRADS)

def adamw(n):
    at = lambda j: [(4 * k + j + 1) << 20 for k in range(n)]
    tl = osa.TensorList(at(0), at(1), m=at(2), v=at(3), weight_decay=[0.0] * n, numel=[8] * n)
    return lambda: osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_ADAMW)

few, many = {"muon": (muon(10), muon(1 << 22)), "grads": (grads(10), grads(1 << 46)), "adamw": (adamw(3), adamw(300000))}[sys.argv[1]]
assert few() > 0
pages = int(open("/proc/self/statm").read().split()[0])
bound = pages * resource.getpagesize() + (48 << 20)  # 48 MiB more than now
before = resource.getrlimit(resource.RLIMIT_AS)
resource.setrlimit(resource.RLIMIT_AS, (bound, before[1]))
try:
    many()
except osa.OptimError as e:
    assert e.code == osa.OPTIM_EINVAL and "memory" in str(e), str(e)
else:
    raise SystemExit("not refused")
assert few() > 0  # the library goes on
resource.setrlimit(resource.RLIMIT_AS, before)
assert many() > 0
print("fine")
"""


@pytest.mark.skipif(not sys.platform.startswith("linux"), reason="bounds the address space through Linux's limits")
@pytest.mark.parametrize("kind", ["muon", "grads", "adamw"])
def test_out_of_host_memory(kind):
    if not os.path.exists(osa.LIB_PATH):
        osa.build_library()
    r = subprocess.run([sys.executable, "-c", PROGRAM, kind], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, (r.returncode, r.stderr[-2000:])
