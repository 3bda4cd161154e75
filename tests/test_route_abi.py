"""Checks of include/optim_route.h and include/optim_dropout.h that need no GPU:
exports, workspace sizes, refusals, the headers from C, and the generator of
csrc/philox.h as constant expressions.  Device pointers are fake integers, never
read: every call here is refused, or has nothing to do."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

import optimizer_step_adamw_amd as osa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40
G = 1 << 30


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(osa.LIB_PATH):
        osa.build_library()
    return osa.lib()


@pytest.mark.parametrize("header,names", [("optim_route.h", osa.EXPORTED_ROUTE), ("optim_dropout.h", osa.EXPORTED_DROPOUT)])
def test_exports(L, header, names):
    text = open(os.path.join(ROOT, "include", header)).read()
    assert set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(optim_\w+)\s*\(", text, re.M)) == set(names)
    for name in names:
        assert hasattr(L, name), name


def route_hp(topk=2, **kw):
    return osa.optim_route_hp(topk, **kw)


def refuses(call, code, cases):
    for kw in cases:
        assert call(**kw) == code, kw
        assert len(osa.lib().optim_last_error().decode()) > 3


def test_route(L):
    def call(x=A, ld=8, dt=osa.OPTIM_F32, t=4, e=8, bias=None, hp=route_hp(), idx=A + G, w=A + 2 * G):
        return L.optim_route(x, ld, dt, t, e, bias, ctypes.byref(hp) if hp else None, idx, w, None)

    assert call(t=0) == call(t=0, x=None, idx=None, w=None) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(x=None), dict(idx=None), dict(w=None), dict(t=-1), dict(e=0), dict(e=1025), dict(ld=7),
                                     dict(ld=1 << 24), dict(hp=None), dict(t=2 ** 30), dict(idx=A), dict(w=A + G), dict(w=A + 4),
                                     dict(bias=A + G)])
    refuses(call, osa.OPTIM_EINVAL, [dict(hp=h) for h in (
        route_hp(0), route_hp(9), route_hp(33), route_hp(score=2), route_hp(score=-1), route_hp(groups=0), route_hp(groups=3),
        route_hp(groups=2, top_groups=0), route_hp(groups=2, top_groups=3), route_hp(groups=2, group_best=3), route_hp(group_best=0),
        route_hp(5, groups=2), route_hp(scale=math.nan), route_hp(scale=math.inf), route_hp(scale=1e39))])
    assert call(e=130, ld=130, hp=route_hp(groups=65)) == osa.OPTIM_EINVAL
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=3), dict(dt=-1)])
    refuses(call, osa.OPTIM_EALIGN, [dict(x=A + 2), dict(idx=A + G + 2), dict(w=A + 2 * G + 1), dict(bias=A + 3 * G + 2),
                                     dict(x=A + 1, dt=osa.OPTIM_BF16)])


def test_route_grad(L):
    def call(x=A, ld=8, dt=osa.OPTIM_F32, t=4, e=8, hp=route_hp(), idx=A + G, dw=A + 2 * G, d=A + 3 * G, ldd=8):
        return L.optim_route_grad(x, ld, dt, t, e, ctypes.byref(hp) if hp else None, idx, dw, d, ldd, None)

    assert call(t=0, x=None, idx=None, dw=None, d=None) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(x=None), dict(idx=None), dict(dw=None), dict(d=None), dict(t=-1), dict(e=0), dict(ld=7),
                                     dict(ldd=7), dict(hp=None), dict(hp=route_hp(0)), dict(d=A), dict(d=A + G), dict(d=A + 2 * G)])
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=7)])
    refuses(call, osa.OPTIM_EALIGN, [dict(x=A + 2), dict(idx=A + G + 1), dict(dw=A + 2 * G + 2), dict(d=A + 3 * G + 2)])


def test_route_bias(L):
    def call(off=A, e=8, bias=A + G, rate=A + 2 * G, found=None):
        return L.optim_step_route_bias(off, e, bias, rate, found, None)

    refuses(call, osa.OPTIM_EINVAL, [dict(off=None), dict(bias=None), dict(rate=None), dict(e=0), dict(e=1025), dict(bias=A), dict(rate=A + G + 4),
                                     dict(found=A + G)])
    refuses(call, osa.OPTIM_EALIGN, [dict(off=A + 2), dict(bias=A + G + 1), dict(rate=A + 2 * G + 2), dict(found=A + 3 * G + 3)])


def test_rows(L):
    out = ctypes.c_size_t(0)
    W = L.optim_route_rows_workspace
    assert W(4, 2, 8, None) == osa.OPTIM_EINVAL
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 33, 8), (4, 2, 0), (4, 2, 1025), (1 << 30, 2, 8), ((1 << 31) - 1, 2, 8)):
        assert W(*bad, ctypes.byref(out)) == osa.OPTIM_EINVAL, bad
    assert W(0, 1, 1, ctypes.byref(out)) == osa.OPTIM_OK and out.value == 0
    assert W(300, 2, 8, ctypes.byref(out)) == osa.OPTIM_OK and out.value == 0
    assert W((1 << 30) - 1, 2, 1024, ctypes.byref(out)) == osa.OPTIM_OK and 0 < out.value < 8 << 20
    need = osa.optim_route_rows_workspace(65536, 8, 256)
    assert need > 0

    def call(idx=A, t=65536, k=8, e=256, off=A + G, place=A + 2 * G, order=A + 3 * G, ws=A + 4 * G, n=need):
        return L.optim_route_rows(idx, t, k, e, off, place, order, ws, n, None)

    refuses(call, osa.OPTIM_EINVAL, [dict(idx=None), dict(off=None), dict(place=None), dict(t=-1), dict(k=0), dict(e=0), dict(place=A),
                                     dict(order=A + 2 * G), dict(off=A + 4), dict(ws=A + 2 * G)])
    refuses(call, osa.OPTIM_EWORKSPACE, [dict(ws=None), dict(n=need - 1), dict(ws=A + 4 * G + 128)])
    refuses(call, osa.OPTIM_EALIGN, [dict(idx=A + 2), dict(off=A + G + 1), dict(place=A + 2 * G + 2), dict(order=A + 3 * G + 1)])


def test_expert_gather(L):
    def call(x=A, ldx=16, dt=osa.OPTIM_BF16, place=A + G, w=None, t=4, k=2, d=16, y=A + 2 * G, ldy=16, rows=8):
        return L.optim_expert_gather(x, ldx, dt, place, w, t, k, d, y, ldy, rows, None)

    assert call(t=0) == call(rows=0) == call(d=0) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(x=None), dict(place=None), dict(y=None), dict(ldx=15), dict(ldy=15), dict(t=-1), dict(k=0),
                                     dict(k=33), dict(d=-1), dict(d=1 << 24), dict(rows=-1), dict(rows=1 << 31), dict(y=A), dict(y=A + G),
                                     dict(w=A + 2 * G), dict(ldx=1 << 24)])
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=9)])
    refuses(call, osa.OPTIM_EALIGN, [dict(x=A + 1), dict(place=A + G + 2), dict(w=A + 3 * G + 2), dict(y=A + 2 * G + 1),
                                     dict(x=A + 2, dt=osa.OPTIM_F32)])


def drop(p=0.5, seed=1, site=0, first=0):
    return osa.optim_dropout_hp(p, seed, site, first)


BAD_DROPS = (drop(-0.1), drop(1.0), drop(math.nan), drop(first=-1), drop(first=(1 << 60) + 1))


def test_expert_combine(L):
    def call(y=A, ldy=16, rows=8, dt=osa.OPTIM_BF16, place=A + G, w=None, t=4, k=2, d=16, res=None, ldr=16, hp=None, step=None,
             out=A + 2 * G, ldo=16):
        return L.optim_expert_combine(y, ldy, rows, dt, place, w, t, k, d, res, ldr, ctypes.byref(hp) if hp else None, step, out, ldo,
                                      None)

    assert call(t=0) == call(d=0) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(y=None), dict(place=None), dict(out=None), dict(ldy=15), dict(ldo=15), dict(res=A + 3 * G, ldr=15),
                                     dict(t=-1), dict(k=0), dict(rows=-1), dict(out=A), dict(out=A + G), dict(res=A + 2 * G, ldr=17),
                                     dict(res=A + 2 * G + 2), dict(hp=drop(), step=A + 2 * G)])
    refuses(call, osa.OPTIM_EINVAL, [dict(hp=h) for h in BAD_DROPS])
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=9)])
    refuses(call, osa.OPTIM_EALIGN, [dict(y=A + 1), dict(place=A + G + 2), dict(w=A + 3 * G + 2), dict(out=A + 2 * G + 1), dict(res=A + 3 * G + 1),
                                     dict(hp=drop(), step=A + 4 * G + 2)])


def test_expert_combine_grad(L):
    def call(do=A, ldd=16, dt=osa.OPTIM_BF16, y=A + G, ldy=16, rows=8, place=A + 2 * G, w=None, t=4, k=2, d=16, hp=None, step=None,
             dy=A + 3 * G, lddy=16, dw=A + 4 * G):
        return L.optim_expert_combine_grad(do, ldd, dt, y, ldy, rows, place, w, t, k, d, ctypes.byref(hp) if hp else None, step, dy, lddy,
                                           dw, None)

    assert call(t=0) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(do=None), dict(y=None), dict(place=None), dict(dy=None, dw=None), dict(ldd=15), dict(ldy=15),
                                     dict(lddy=15), dict(t=-1), dict(k=0), dict(rows=-1), dict(d=-1), dict(dy=A), dict(dy=A + G, lddy=17),
                                     dict(dy=A + G + 2), dict(dw=A), dict(dw=A + 2 * G), dict(dw=A + 3 * G), dict(w=A + 4 * G)])
    refuses(call, osa.OPTIM_EINVAL, [dict(hp=h) for h in BAD_DROPS])
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=-3)])
    refuses(call, osa.OPTIM_EALIGN, [dict(do=A + 1), dict(y=A + G + 1), dict(place=A + 2 * G + 2), dict(w=A + 5 * G + 2), dict(dy=A + 3 * G + 1),
                                     dict(dw=A + 4 * G + 2)])


def test_dropout(L):
    def call(x=A, dt=osa.OPTIM_F32, n=100, res=None, hp=drop(), step=None, out=A + G):
        return L.optim_dropout(x, dt, n, res, ctypes.byref(hp) if hp else None, step, out, None)

    assert call(n=0) == call(n=0, x=None, out=None) == osa.OPTIM_OK
    refuses(call, osa.OPTIM_EINVAL, [dict(x=None), dict(out=None), dict(hp=None), dict(n=-1), dict(n=(1 << 48) + 1), dict(out=A + 4),
                                     dict(res=A + G + 4), dict(step=A + G)])
    refuses(call, osa.OPTIM_EINVAL, [dict(hp=h) for h in BAD_DROPS])
    refuses(call, osa.OPTIM_EDTYPE, [dict(dt=9)])
    refuses(call, osa.OPTIM_EALIGN, [dict(x=A + 2), dict(out=A + G + 2), dict(res=A + 2 * G + 2), dict(step=A + 2 * G + 2)])


def test_binding_refuses(L):
    import torch
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(9, dtype=torch.int32)
    for call in (lambda: osa.optim_route(f.double(), route_hp(), i, torch.zeros(4, 2)),
                 lambda: osa.optim_route(f, route_hp(), i, torch.zeros(4, 2)),  # not on a GPU
                 lambda: osa.optim_route_grad(f, route_hp(), i, torch.zeros(4, 2), f.bfloat16()),
                 lambda: osa.optim_route_rows(i.long(), off, i),
                 lambda: osa.optim_route_rows(i, off, i[:2]),
                 lambda: osa.optim_step_route_bias(off, torch.zeros(9), torch.zeros(1)),
                 lambda: osa.optim_expert_gather(f, i, torch.zeros(8, 9)),
                 lambda: osa.optim_expert_gather(f, i, torch.zeros(8, 8).half()),
                 lambda: osa.optim_expert_combine(torch.zeros(8, 8), i, torch.zeros(5, 8)),
                 lambda: osa.optim_expert_combine_grad(f, None, i, None),
                 lambda: osa.optim_expert_combine_grad(f, None, i, torch.zeros(8, 8), dweights=torch.zeros(4, 2)),
                 lambda: osa.optim_dropout(f, f[:2], drop()),
                 lambda: osa.optim_dropout(f, f, drop(), step=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


PROGRAM = r"""
#include "optim_route.h"
#include <stdio.h>

int main(void) {
    optim_route_hp hp = {8, OPTIM_ROUTE_SIGMOID, 1, 8, 4, 2, 2.5};
    optim_dropout_hp drop = {0.1, 7, 0, 3};
    size_t bytes = 0;
    int rc = optim_route_rows_workspace(65536, 8, 256, &bytes);
    printf("rows %d %zu\n", rc, bytes);
    rc = optim_route(NULL, 256, OPTIM_F32, 4, 256, NULL, &hp, NULL, NULL, NULL);
    printf("route %d\n", rc);
    rc = optim_dropout(NULL, OPTIM_F16, 0, NULL, &drop, NULL, NULL, NULL);
    printf("dropout %d\n", rc);
    printf("sizes %zu %zu\n", sizeof hp, sizeof drop);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not found")
def test_headers_compile_as_c_and_match_the_binding(L, tmp_path):
    src, exe, libdir = tmp_path / "abi.c", tmp_path / "abi", os.path.dirname(osa.LIB_PATH)
    src.write_text(PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-L", libdir, "-l:liboptim_step.so", f"-Wl,-rpath,{libdir}", "-Wl,-rpath-link,/opt/rocm/lib"], check=True,
                   capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout.split("\n")
    rows = {r.split()[0]: r.split()[1:] for r in out if r.strip()}
    assert rows["rows"] == ["0", str(osa.optim_route_rows_workspace(65536, 8, 256))]
    assert rows["route"] == [str(osa.OPTIM_EINVAL)] and rows["dropout"] == ["0"]
    assert rows["sizes"] == [str(ctypes.sizeof(osa.optim_route_hp)), str(ctypes.sizeof(osa.optim_dropout_hp))]


# The first two lines are the generator's published known answers.
GENERATOR = r"""
#include "philox.h"
using namespace optim;
constexpr bool same(Words x, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return x.w[0] == a && x.w[1] == b && x.w[2] == c && x.w[3] == d;
}
static_assert(same(philox(0, 0, 0, 0), 0x6627e8d5u, 0xe169c58du, 0xbc57ac4cu, 0x9b00dbd8u), "zeros");
static_assert(same(philox(~0ull, ~0u, ~0u, ~0ull), 0x408f276du, 0x41c83b0eu, 0xa20bc7c6u, 0x6d5451fdu), "ones");
// eight draws from any place on are those of the blocks they lie in
constexpr bool places(uint64_t q0) {
    for (uint64_t q = q0; q < q0 + 20; ++q) {
        const Words got = draws8(q, 5, 9, 77);
        for (int i = 0; i < 8; ++i) {
            const uint64_t at = q + i;
            if (draw_of(got, i) != draw_of(philox(at >> 3, 5, 9, 77), (int)(at & 7))) return false;
        }
    }
    return true;
}
static_assert(places(0) && places((1ull << 35) - 9) && places((1ull << 60) - 9), "places");
int main() { return 0; }
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_the_generator(tmp_path):
    src = tmp_path / "philox.cpp"
    src.write_text(GENERATOR)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-fconstexpr-ops-limit=100000000", "-I",
                        os.path.join(ROOT, "optimizer_step_adamw_amd", "csrc"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
