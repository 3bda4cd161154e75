"""Norms of gradient lists and clipping in place (include/optim_grads.h)
against float64: every type and kind of norm, ragged and misaligned buckets,
empty tensors, values whose squares leave fp32's range, NaN / Inf, bars that
clip and bars that do not, several lists under one norm, the static
workspace, other streams and graph replays.

Tolerances: a norm is summed in fp64 over fp32 sums of at most 8 positive
terms, each rounding at most 2^-24 of its result, and rounded once to fp32:
9 * 2^-24 relative (L1; half of the sum's part for L2; none for INF but the
product with inv_scale).  The factor adds the same again, in fp64, and one
rounding.  Clipped gradients equal one fp32 product rounded to the type, bit
for bit."""
import math

import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DEV, say

pytestmark = pytest.mark.gpu

KINDS = {"l2": osa.OPTIM_NORM_L2, "l1": osa.OPTIM_NORM_L1, "inf": osa.OPTIM_NORM_INF}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOL = 9 * 2.0 ** -24
# one element, both sides of the vector width, of a bundle's limit and of an item's
RAGGED = [1, 0, 3, 7, 8, 9, 255, 4095, 4096, 4097, 0, 32767, 32768, 32769, 100003, 5, 65536, 131073, 2]


def bucket(sizes, dtype, std, seed, shift=0):
    """Tensors end to end in one buffer, `shift` elements behind a boundary."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    flat = (torch.randn(sum(sizes) + shift, generator=gen, device=DEV, dtype=torch.float64) * std).to(dtype)
    return flat, list(flat[shift:].split(sizes))


def norm64(x, kind):
    x = x.double().abs()
    if x.numel() == 0:
        return 0.0
    return float({"l2": lambda: x.square().sum().sqrt(), "l1": x.sum, "inf": x.max}[kind]())


def whole64(norms, kind):
    return {"l2": lambda: math.sqrt(math.fsum(v * v for v in norms)), "l1": lambda: math.fsum(norms),
            "inf": lambda: max(norms, default=0.0)}[kind]()


class Out:
    def __init__(self, n):
        # sentinels: what a call must overwrite
        self.norms = torch.full((n,), -7.0, device=DEV)
        self.total, self.coef, self.found = (torch.full((1,), v, device=DEV) for v in (-7.0, -7.0, 0.0))

    def args(self):
        return self.found, self.norms, self.total, self.coef


def check_norms(out, grads, kind, s, max_norm, what):
    want = [abs(s) * norm64(g, kind) for g in grads]
    got = out.norms.tolist()
    for i, (a, b) in enumerate(zip(got, want)):
        assert abs(a - b) <= TOL * b, (what, i, a, b)
    total = whole64(want, kind)
    assert abs(out.total.item() - total) <= TOL * total, (what, out.total.item(), total)
    c = s * (min(1.0, max_norm / (total + 1e-6)) if 0 < max_norm < math.inf else 1.0)
    assert abs(out.coef.item() - c) <= 2 * TOL * abs(c), (what, out.coef.item(), c)


@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norms_and_clip_of_a_ragged_bucket(dtype, kind, shift):
    say(dtype, kind, shift)
    flat, grads = bucket(RAGGED, DTYPES[dtype], 3.0, 11 + shift, shift)
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    s = 0.125
    inv = torch.tensor([s], device=DEV)
    total = whole64([s * norm64(g, kind) for g in grads], kind)
    for max_norm in (0.3 * total, 2.0 * total, 0.0, -1.0, math.inf):
        out = Out(len(grads))
        before = flat.clone()
        osa.optim_grad_norms(plan.handle, KINDS[kind], inv, max_norm, *out.args())
        check_norms(out, grads, kind, s, max_norm, (dtype, kind, shift, max_norm))
        assert out.found.item() == 0.0
        assert torch.equal(flat, before)
    # the last bar leaves s alone; clip with a factor below it
    osa.optim_grad_norms(plan.handle, KINDS[kind], inv, 0.3 * total, *out.args())
    osa.optim_clip_grads(plan.handle, out.coef, out.found)
    want = before.clone()
    want[shift:] = (before[shift:].float() * out.coef).to(flat.dtype)
    assert torch.equal(flat.view(torch.uint8), want.view(torch.uint8))
    # the clipped gradients' norm is the bar, up to each element's rounding to its type
    again = Out(len(grads))
    osa.optim_grad_norms(plan.handle, KINDS[kind], None, 0.0, *again.args())
    check_norms(again, grads, kind, 1.0, 0.0, "again")
    if dtype != "f16":  # (fp16's subnormals round by more than half a step relative)
        assert abs(again.total.item() - 0.3 * total) <= (torch.finfo(flat.dtype).eps / 2 + 2 * TOL) * 0.3 * total + 1e-6


def test_factor_of_one_and_overflow_leave_the_gradients():
    flat, grads = bucket([5000, 33], torch.float32, 1.0, 5)
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    before = flat.clone()
    one, half, zero = (torch.tensor([v], device=DEV) for v in (1.0, 0.5, 0.0))
    osa.optim_clip_grads(plan.handle, one)
    osa.optim_clip_grads(plan.handle, half, one)  # found_inf set
    assert torch.equal(flat, before)
    osa.optim_clip_grads(plan.handle, half, zero)
    assert torch.equal(flat, before * 0.5)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("value", [1e-30, 1e-20, 1e25, 1e30])
def test_magnitudes_beyond_fp32_squares(value, kind):
    flat, grads = bucket([300, 70000, 4097], torch.float32, value, 23)
    grads[0].zero_()
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    out = Out(3)
    osa.optim_grad_norms(plan.handle, KINDS[kind], None, 0.0, *out.args())
    check_norms(out, grads, kind, 1.0, 0.0, (value, kind))
    assert out.found.item() == 0.0


@pytest.mark.parametrize("where", [0, 299, 300, 36000, 70299])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_non_finite(dtype, kind, bad, where):
    flat, grads = bucket([300, 70000], DTYPES[dtype], 1.0, 31)
    flat[where] = bad
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    out, inv = Out(2), torch.tensor([0.5], device=DEV)
    osa.optim_grad_norms(plan.handle, KINDS[kind], inv, 1e-3, *out.args())
    hit, other = (0, 1) if where < 300 else (1, 0)
    got = out.norms.tolist()
    same = (lambda v: math.isnan(v)) if math.isnan(bad) else (lambda v: v == math.inf)
    assert same(got[hit]) and same(out.total.item()), (got, out.total.item())
    want = 0.5 * norm64(grads[other], kind)
    assert abs(got[other] - want) <= TOL * want
    assert out.found.item() == 1.0 and out.coef.item() == 0.5


def test_many_tiny_tensors_and_optional_outputs():
    sizes = [1 + (k * 7919) % 700 for k in range(6001)]
    flat, grads = bucket(sizes, torch.bfloat16, 1.0, 41)
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    out = Out(len(sizes))
    osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, None, 1.0, *out.args())
    want = torch.stack([g.double().square().sum().sqrt() for g in grads])
    assert ((out.norms - want).abs() <= TOL * want).all()
    alone = torch.zeros(1, device=DEV)
    osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, None, 1.0, None, None, alone, None)
    assert alone.item() == out.total.item()


@pytest.mark.parametrize("sizes", [[], [0], [0, 0, 0]])
def test_empty_lists(sizes):
    grads = [torch.empty(n, device=DEV) for n in sizes]
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    out, inv = Out(len(sizes)), torch.tensor([0.25], device=DEV)
    for kind in KINDS.values():
        osa.optim_grad_norms(plan.handle, kind, inv, 1.0, *out.args())
        osa.optim_clip_grads(plan.handle, out.coef)
        assert out.total.item() == 0.0 and out.coef.item() == 0.25 and all(v == 0.0 for v in out.norms.tolist())


@pytest.mark.parametrize("kind", list(KINDS))
def test_one_norm_over_several_lists(kind):
    _, a = bucket([5000, 77], torch.float32, 1.0, 51)
    _, b = bucket([40000, 3], torch.bfloat16, 2.0, 52)
    plans = [osa.Plan(osa.grad_list(g), osa.OPTIM_ALGO_GRADS) for g in (a, b)]
    totals, inv = torch.zeros(3, device=DEV), torch.tensor([0.5], device=DEV)
    for k, plan in enumerate(plans):
        osa.optim_grad_norms(plan.handle, KINDS[kind], inv, 0.0, None, None, totals[k:k + 1], None)
    want = whole64([0.5 * norm64(g, kind) for g in a + b], kind)
    coef = torch.zeros(1, device=DEV)
    osa.optim_clip_coef(totals, 2, KINDS[kind], inv, 0.1 * want, totals[2:], coef)
    assert abs(totals[2].item() - want) <= 2 * TOL * want
    assert abs(coef.item() - 0.5 * 0.1 * want / (want + 1e-6)) <= 4 * TOL * coef.item()
    # in place over the list, none at all, and NaN / Inf
    osa.optim_clip_coef(totals, 2, KINDS[kind], None, 0.1 * want, totals[:1], None)
    assert totals[0].item() == totals[2].item()
    osa.optim_clip_coef(None, 0, KINDS[kind], inv, 1.0, totals[:1], coef)
    assert totals[0].item() == 0.0 and coef.item() == 0.5
    for bad in (math.nan, math.inf):
        v = torch.tensor([1.0, bad, 2.0], device=DEV)
        osa.optim_clip_coef(v, 3, KINDS[kind], inv, 1.0, totals[:1], coef)
        assert (math.isnan(totals[0].item()) if math.isnan(bad) else totals[0].item() == math.inf) and coef.item() == 0.5


def test_repeats_bit_for_bit_on_another_stream_and_the_static_workspace():
    _, grads = bucket([1 << 20, 17, 300001], torch.bfloat16, 1.0, 61)
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    ref = Out(3)
    osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, None, 1.0, *ref.args())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        out = Out(3)
        side.wait_stream(torch.cuda.current_stream())
        osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, None, 1.0, *out.args(), stream=side)
        side.synchronize()
        assert torch.equal(out.norms, ref.norms) and torch.equal(out.total, ref.total) and torch.equal(out.coef, ref.coef)
    h = osa.optim_plan_create_static(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS, None)
    out = Out(3)
    osa.optim_grad_norms(h, osa.OPTIM_NORM_L2, None, 1.0, *out.args())
    assert torch.equal(out.norms, ref.norms) and torch.equal(out.total, ref.total)
    osa.optim_plan_destroy(h)


def test_captured_and_replayed():
    flat, grads = bucket([4096, 33, 200001, 1], torch.float32, 1.0, 71)
    twin = flat.clone()
    tgrads = list(twin.split([4096, 33, 200001, 1]))
    plan, tplan = (osa.Plan(osa.grad_list(g), osa.OPTIM_ALGO_GRADS) for g in (grads, tgrads))
    out, tout = Out(4), Out(4)

    def once(p, o):
        osa.optim_grad_norms(p.handle, osa.OPTIM_NORM_L2, None, 100.0, *o.args())
        osa.optim_clip_grads(p.handle, o.coef, o.found)

    torch.cuda.synchronize()
    cs, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        with torch.cuda.graph(g, stream=cs):
            once(plan, out)
    torch.cuda.current_stream().wait_stream(cs)
    for k in range(5):
        fresh = torch.randn_like(flat) * (k + 0.1)
        flat.copy_(fresh)
        twin.copy_(fresh)
        g.replay()
        once(tplan, tout)
        torch.cuda.synchronize()
        for a, b in ((flat, twin), (out.norms, tout.norms), (out.total, tout.total), (out.coef, tout.coef)):
            assert torch.equal(a, b), k


def test_a_tensor_past_2_31_elements():
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[n - 3:] = 4.0
    g[12345] = 3.0
    plan = osa.Plan(osa.grad_list([g]), osa.OPTIM_ALGO_GRADS)
    out = Out(1)
    osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_L2, None, 1.0, *out.args())
    want = math.sqrt(3 * 16 + 9)
    assert abs(out.total.item() - want) <= TOL * want
    osa.optim_clip_grads(plan.handle, torch.tensor([0.5], device=DEV))
    assert g[n - 3:].tolist() == [2.0] * 3 and g[12345].item() == 1.5 and float(g[-70000:-3].abs().max()) == 0.0


def test_trace_names_the_kernels():
    _, grads = bucket([70000], torch.float16, 1.0, 81)
    plan = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    osa.optim_plan_trace(plan.handle, 8)
    out = Out(1)
    osa.optim_grad_norms(plan.handle, osa.OPTIM_NORM_INF, None, 1.0, *out.args())
    osa.optim_clip_grads(plan.handle, out.coef)
    recs, dropped = osa.optim_plan_trace_read(plan.handle)
    assert [(k, w) for k, w, _ in recs] == [("grad_norms_kernel", 3), ("clip_grads_kernel", 3)] and dropped == 0
