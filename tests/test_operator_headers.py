"""include/optim_grads.h and include/optim_muon.h from C: a C99 program (gcc,
-Wall -Wextra -Werror) includes both, sizes a plan of each kind, asks for an
expert workspace and reads refusals.  Struct sizes and results must agree with
the Python binding's.  No device is touched."""
import ctypes
import os
import shutil
import subprocess

import pytest

import optimizer_step_adamw_amd as osa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "optim_grads.h"
#include "optim_muon.h"
#include <stdio.h>
#include <string.h>

int main(void) {
    int64_t numel[2] = {600000, 77}, rows[2] = {300, 7}, cols[2] = {200, 11};
    uintptr_t base = (uintptr_t)1 << 40;
    void *p[2], *g[2], *m[2];
    double wd[2] = {0.1, 0.0};
    for (int i = 0; i < 2; ++i) {
        p[i] = (void *)(base + (uintptr_t)(3 * i + 0) * (1u << 24));
        g[i] = (void *)(base + (uintptr_t)(3 * i + 1) * (1u << 24));
        m[i] = (void *)(base + (uintptr_t)(3 * i + 2) * (1u << 24));
    }
    optim_tensor_list tl;
    memset(&tl, 0, sizeof tl);
    tl.n = 2;
    tl.numel = numel;
    tl.grad = (const void *const *)g;
    tl.grad_dtype = OPTIM_F16;
    size_t bytes = 0;
    int rc = optim_plan_workspace_size(&tl, OPTIM_ALGO_GRADS, NULL, &bytes);
    printf("grads %d %zu\n", rc, bytes);
    tl.param = p;
    tl.m = m;
    tl.weight_decay = wd;
    tl.grad_dtype = OPTIM_F32;
    tl.param_dtype = OPTIM_F32;
    tl.rows = rows;
    tl.cols = cols;
    rc = optim_plan_workspace_size(&tl, OPTIM_ALGO_MUON, NULL, &bytes);
    printf("muon %d %zu\n", rc, bytes);
    rc = optim_expert_grad_workspace(2, 8192, 128, 64, &bytes);
    printf("expert %d %zu\n", rc, bytes);
    optim_muon_hp hp = {0.95, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, OPTIM_MUON_SCALE_RMS};
    rc = optim_step_muon(NULL, &hp, NULL, NULL, NULL, NULL, NULL);
    printf("refused %d %d\n", rc, (int)(strlen(optim_last_error()) > 0));
    rc = optim_clip_coef(NULL, 3, OPTIM_NORM_L1, NULL, 1.0, NULL, NULL, NULL);
    printf("coef %d\n", rc);
    printf("sizes %zu %zu\n", sizeof(optim_tensor_list), sizeof hp);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not found")
def test_headers_compile_as_c_and_match_the_binding(tmp_path):
    lib = osa.LIB_PATH
    if not os.path.exists(lib):
        pytest.skip("library not built")
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text(PROGRAM)
    libdir = os.path.dirname(lib)
    cmd = ["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
           "-o", str(exe), "-L", libdir, "-l:liboptim_step.so", f"-Wl,-rpath,{libdir}",
           "-Wl,-rpath-link,/opt/rocm/lib"]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout.split("\n")
    rows = {r.split()[0]: r.split()[1:] for r in out if r.strip()}
    at = lambda j: [(1 << 40) + (3 * i + j) * (1 << 24) for i in range(2)]  # noqa: E731
    numel = [600000, 77]
    gl = osa.TensorList([None, None], at(1), weight_decay=[0.0, 0.0], numel=numel, grad_dtype=osa.OPTIM_F16)
    grads = osa.optim_plan_workspace_size(gl, osa.OPTIM_ALGO_GRADS)
    assert rows["grads"] == ["0", str(grads)]
    tl = osa.TensorList(at(0), at(1), m=at(2), weight_decay=[0.1, 0.0], numel=numel, rows=[300, 7], cols=[200, 11])
    assert rows["muon"] == ["0", str(osa.optim_plan_workspace_size(tl, osa.OPTIM_ALGO_MUON))]
    assert rows["expert"] == ["0", str(osa.optim_expert_grad_workspace(2, 8192, 128, 64))]
    assert rows["refused"] == [str(osa.OPTIM_EINVAL), "1"] and rows["coef"] == [str(osa.OPTIM_EINVAL)]
    assert rows["sizes"] == [str(ctypes.sizeof(osa.optim_tensor_list)), str(ctypes.sizeof(osa.optim_muon_hp))]
