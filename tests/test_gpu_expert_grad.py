"""Experts' weight gradients (optim_expert_grad) against float64: both input
and output types, ragged and empty runs, rows outside every run, odd sizes,
strides and alignments, accumulation, sums in one piece and in several.

Tolerance, element by element: products of two 16-bit numbers are exact in
fp32, and each of the k additions of a run is off by at most a whole step of
fp32 (2^-23) of the sum of magnitudes: k 2^-23 sum |x| |y|; the product with
the scale, the accumulation and the rounding to the output's type add half a
step each of the values they produce."""
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, say

pytestmark = pytest.mark.gpu

# (runs, m, n): whole tiles and steps, odd ones, sides of one, runs of 0, 1, 63, 64, 65, 200
CASES = [([64, 128], 128, 128), ([0, 1, 63, 64, 65, 200, 0], 136, 264), ([300], 256, 172), ([5, 0, 70], 1, 1),
         ([130, 7], 33, 200), ([64, 3], 7, 5), ([129], 300, 131), ([0, 0], 64, 64), ([1000], 72, 40), ([40, 41], 129, 257)]


def make(runs, m, n, dtype, out, before=0, behind=0, padx=0, pady=0, shift=0, seed=1):
    """x and dy of `before` + sum(runs) + `behind` rows, `pad` elements between rows, `shift` behind a boundary; what lies
    outside the runs and between the rows is NaN."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = before + sum(runs) + behind

    def matrix(w, pad):
        whole = torch.full((shift + t * (w + pad) + 8,), float("nan"), dtype=dtype, device=DEV)
        v = whole[shift:shift + t * (w + pad)].view(t, w + pad)[:, :w]
        v[before:t - behind if behind else t] = torch.randn(sum(runs), w, generator=gen, device=DEV).to(dtype)
        return v

    off = [before]
    for r in runs:
        off.append(off[-1] + r)
    dw = torch.randn(len(runs), m, n, generator=gen, device=DEV).to(out)
    return matrix(m, padx), matrix(n, pady), torch.tensor(off, dtype=torch.int32, device=DEV), dw, off


def check(x, y, off, before, dw, accumulate, scale):
    for e in range(dw.shape[0]):
        a, b = x[off[e]:off[e + 1]].double(), y[off[e]:off[e + 1]].double()
        want = a.t().contiguous() @ b * scale
        size = a.abs().t().contiguous() @ b.abs() * abs(scale)
        if accumulate:
            want = want + before[e].double()
        step = torch.finfo(dw.dtype).eps / 2
        room = (a.shape[0] + 1) * 2.0 ** -23 * size + (2.0 ** -23 + step) * want.abs() + 1e-38
        off_by = (dw[e].double() - want).abs()
        assert (off_by <= room).all(), (e, float((off_by - room).max()))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("runs,m,n", CASES)
def test_runs(runs, m, n, dtype, out, accumulate):
    say(runs, m, n, dtype, out, accumulate)
    scale = torch.tensor([0.5], device=DEV)
    for kw in ({}, dict(before=3, behind=5), dict(padx=8, pady=24), dict(padx=1, pady=3, shift=1), dict(shift=4)):
        x, y, o, dw, off = make(runs, m, n, dtype, out, **kw)
        old = dw.clone()
        osa.optim_expert_grad(x, y, o, dw, accumulate=accumulate, scale=scale)
        check(x, y, off, old, dw, accumulate, 0.5)


@pytest.mark.parametrize("runs,m,n", [([5000], 136, 264), ([700, 0, 4100], 130, 67), ([8192, 0, 0, 64], 256, 128)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_in_pieces(runs, m, n, out, accumulate):
    x, y, o, dw, off = make(runs, m, n, torch.bfloat16, out, before=2, behind=1)
    nbytes = osa.optim_expert_grad_workspace(len(runs), x.shape[0], m, n)
    pieces = nbytes // (len(runs) * m * n * 4)
    assert pieces > 1 and nbytes % (len(runs) * m * n * 4) == 0
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN
    old, twin = dw.clone(), dw.clone()
    osa.optim_expert_grad(x, y, o, dw, accumulate=accumulate, workspace=ws)
    check(x, y, off, old, dw, accumulate, 1.0)
    osa.optim_expert_grad(x, y, o, twin, accumulate=accumulate, workspace=ws)
    assert torch.equal(dw, twin)  # the same bits again
    with pytest.raises(osa.OptimError) as ei:
        osa.optim_expert_grad(x, y, o, dw, accumulate=accumulate, workspace=ws[:256])
    assert ei.value.code == osa.OPTIM_EWORKSPACE


def test_bounds_are_clamped():
    """Offsets beyond the rows or decreasing: runs inside [0, tokens] only."""
    x, y, _, dw, _ = make([100], 64, 64, torch.bfloat16, torch.float32)
    dw = torch.full((4, 64, 64), 7.0, device=DEV)
    o = torch.tensor([-50, 40, 20, 1 << 30, 60], dtype=torch.int32, device=DEV)
    osa.optim_expert_grad(x, y, o, dw)
    # runs: [0, 40), [40, 40), [20, 100), [100, 100)
    check(x, y, [0, 40], None, dw[:1], False, 1.0)
    check(x, y, [20, 100], None, dw[2:3], False, 1.0)
    assert float(dw[1].abs().max()) == 0.0 and float(dw[3].abs().max()) == 0.0


def test_nothing_to_do():
    x = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    dw = torch.ones(3, 16, 24, device=DEV)
    o = torch.zeros(4, dtype=torch.int32, device=DEV)
    osa.optim_expert_grad(x, y, o, dw, accumulate=True)
    assert torch.equal(dw, torch.ones_like(dw))
    osa.optim_expert_grad(x, y, o, dw)
    assert torch.equal(dw, torch.zeros_like(dw))
    osa.optim_expert_grad(x, y, o[:1], dw[:0])


def test_gradient_of_the_layer_against_autograd_and_differences():
    """dW of sum(c * (x W_e)) by the formula, by autograd in float64 and by a central difference."""
    runs, m, n = [70, 0, 33], 24, 40
    x, _, o, dw, off = make(runs, m, n, torch.bfloat16, torch.float32)
    c = torch.randn(sum(runs), n, device=DEV).to(torch.bfloat16)
    osa.optim_expert_grad(x, c, o, dw)
    w = torch.randn(3, m, n, dtype=torch.float64, device=DEV, requires_grad=True)

    def loss(w):
        return sum((c[a:b].double() * (x[a:b].double() @ w[e])).sum() for e, (a, b) in enumerate(zip(off, off[1:])))

    loss(w).backward()
    assert torch.allclose(dw.double(), w.grad, rtol=0, atol=float(71 * 2.0 ** -23 * 71 * 16))
    d = torch.randn_like(w)
    with torch.no_grad():
        diff = (loss(w + 1e-3 * d) - loss(w - 1e-3 * d)) / 2e-3  # the loss is linear in W
        assert abs(float((dw.double() * d).sum() - diff)) <= 1e-5 * float((w.grad.abs() * d.abs()).sum())


def test_two_streams_and_replays():
    a = make([200, 33, 0, 500], 136, 72, torch.bfloat16, torch.float32, seed=3)
    b = make([65, 1, 900], 40, 264, torch.float16, torch.bfloat16, seed=4)
    refs = []
    for x, y, o, dw, _ in (a, b):
        refs.append(dw.clone())
        osa.optim_expert_grad(x, y, o, refs[-1], accumulate=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [dw.clone() for _, _, _, dw, _ in (a, b)]
    torch.cuda.synchronize()
    for s, (x, y, o, _, _), g in zip(streams, (a, b), got):
        osa.optim_expert_grad(x, y, o, g, accumulate=True, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(got, refs))
    x, y, o, dw, off = a
    ws = torch.empty(max(256, osa.optim_expert_grad_workspace(4, x.shape[0], 136, 72)), dtype=torch.uint8, device=DEV)
    out, twin = dw.clone(), dw.clone()
    torch.cuda.synchronize()
    cs, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        with torch.cuda.graph(g, stream=cs):
            osa.optim_expert_grad(x, y, o, out, accumulate=True, workspace=ws)
    torch.cuda.current_stream().wait_stream(cs)
    for k in range(4):
        o.copy_(torch.tensor([0, 50 + k, 60, 60, 700 + k], dtype=torch.int32))  # another routing
        g.replay()
        torch.cuda.synchronize()
        osa.optim_expert_grad(x, y, o, twin, accumulate=True, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, twin), k


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32, and elements of dW past 2^31."""
    t, m = (1 << 19) + 100, 8192
    x = torch.zeros(t, m, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(t, 8, dtype=torch.bfloat16, device=DEV)
    x[t - 70:, :] = 2.0
    y[t - 70:, :] = 1.0
    dw = torch.full((2, m, 8), 5.0, device=DEV)
    o = torch.tensor([0, t - 100, t], dtype=torch.int32, device=DEV)
    osa.optim_expert_grad(x, y, o, dw)
    assert float(dw[0].abs().max()) == 0.0 and bool((dw[1] == 140.0).all())
    del x, y, dw
    torch.cuda.empty_cache()
    e, m, n = 260, 2896, 2896  # 2.18e9 elements
    dw = torch.full((e, m, n), 3.0, dtype=torch.bfloat16, device=DEV)
    x, y = torch.ones(64, m, dtype=torch.bfloat16, device=DEV), torch.ones(64, n, dtype=torch.bfloat16, device=DEV)
    o = torch.full((e + 1,), 64, dtype=torch.int32, device=DEV)
    o[:e] = 0
    osa.optim_expert_grad(x, y, o, dw)
    assert bool((dw[e - 1] == 64.0).all()) and float(dw[:e - 1].abs().max()) == 0.0


def test_binding_refusals():
    x, y, o, dw, _ = make([64], 32, 48, torch.bfloat16, torch.float32)
    bad = [lambda: osa.optim_expert_grad(x, y.half(), o, dw), lambda: osa.optim_expert_grad(x, y, o.long(), dw),
           lambda: osa.optim_expert_grad(x, y[:-1], o, dw), lambda: osa.optim_expert_grad(x, y, o, dw[:, :, :-1]),
           lambda: osa.optim_expert_grad(x.t(), y, o, dw), lambda: osa.optim_expert_grad(x.cpu(), y, o, dw),
           lambda: osa.optim_expert_grad(x, y, o, dw.transpose(1, 2)), lambda: osa.optim_expert_grad(x.float(), y.float(), o, dw),
           lambda: osa.optim_expert_grad(x, y, o, dw.double())]
    for fn in bad:
        with pytest.raises((ValueError, osa.OptimError)):
            fn()
    with pytest.raises(osa.OptimError) as ei:  # dW over X
        osa.optim_expert_grad(x, y, o, x.reshape(-1)[:32 * 48].view(1, 32, 48))
    assert ei.value.code == osa.OPTIM_EINVAL
