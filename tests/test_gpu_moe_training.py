"""A layer of experts trained with all of its operators together: routing by
groups with a balance bias, the experts' rows, tokens to them and back with
dropout onto the residual, the weight gradients, the router's gradient, the
bias' step and AdamW's; and the chain without the experts' products captured in
a HIP graph.

Against a float64 model on the host that takes each iteration's parameters as
they are on the GPU, with the choices and masks of the definitions: the choice
has to be the same, the output within bf16's half step of the sums (2^-8 of the
terms' magnitudes, three roundings: the rows', the experts' and the output's),
gradients within 3 * 2^-8 of their norm, the roundings of the rows to bf16 (out,
back, and through the product) that lie before each."""
import numpy as np
import pytest
import torch

import optimizer_step_adamw_amd as osa
from gpu_support import DevScalars
from route_support import DEV, f64, kept, route, route_grad, rows_of

pytestmark = pytest.mark.gpu

T, D, E, K = 96, 48, 16, 3
HP = osa.optim_route_hp(K, osa.OPTIM_ROUTE_SIGMOID, 1, 4, 2, 2, 1.5)


def test_a_training_loop_of_a_layer():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device=DEV) * std  # noqa: E731
    w, router, bias = rnd(E, D, D, std=0.2), rnd(D, E, std=0.3), torch.zeros(E, device=DEV)
    gw, gr = torch.zeros_like(w), torch.zeros_like(router)
    m, v = ([torch.zeros_like(p) for p in (w, router)] for _ in range(2))
    adam = osa.Plan(osa.TensorList([w, router], [gw, gr], m=m, v=v, weight_decay=[0.0, 0.0]), osa.OPTIM_ALGO_ADAMW)
    sc, rate = DevScalars(1e-3), torch.tensor([1e-2], device=DEV)
    drop = osa.optim_dropout_hp(0.2, 99, 4)
    idx, wt = torch.empty(T, K, dtype=torch.int32, device=DEV), torch.empty(T, K, device=DEV)
    off, place = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T, K, dtype=torch.int32, device=DEV)
    logits, dlogits, dwt = torch.empty(T, E, device=DEV), torch.empty(T, E, device=DEV), torch.empty(T, K, device=DEV)
    for it in range(3):
        x, res, dout = (rnd(T, D).to(torch.bfloat16) for _ in range(3))
        padded = slice(T - 10, T)  # the batch's end goes nowhere
        w16 = w.to(torch.bfloat16)
        torch.mm(x.float(), router, out=logits)
        logits[padded] = -np.inf
        b64 = f64(bias)
        # forward
        osa.optim_route(logits, HP, idx, wt, bias=bias)
        osa.optim_route_rows(idx, off, place)
        rows = torch.zeros(T * K, D, dtype=torch.bfloat16, device=DEV)
        osa.optim_expert_gather(x, place, rows)
        o = off.tolist()
        y = torch.zeros_like(rows)
        for e in range(E):
            y[o[e]:o[e + 1]] = (rows[o[e]:o[e + 1]].float() @ w16[e].float()).to(torch.bfloat16)
        out = torch.empty_like(x)
        osa.optim_expert_combine(y, place, out, weights=wt, residual=res, dropout=drop, step=sc.step)
        # backward
        dy, dx = torch.zeros_like(y), torch.empty_like(x)
        osa.optim_expert_combine_grad(dout, y, place, dy, weights=wt, dweights=dwt, dropout=drop, step=sc.step)
        osa.optim_expert_grad(rows, dy, off, gw)
        drows = torch.zeros_like(rows)
        for e in range(E):
            drows[o[e]:o[e + 1]] = (dy[o[e]:o[e + 1]].float() @ w16[e].float().t()).to(torch.bfloat16)
        osa.optim_expert_combine(drows, place, dx)
        osa.optim_route_grad(logits, HP, idx, dwt, dlogits)
        torch.mm(x.float().t(), dlogits, out=gr)
        torch.cuda.synchronize()

        # ---- the same on the host
        l64, x64, w64 = f64(logits), f64(x), f64(w16)
        want_idx, wt64 = route(l64, b64, HP)
        assert np.array_equal(idx.cpu().numpy(), want_idx) and (want_idx[padded] == -1).all() and (want_idx[:T - 10] >= 0).all()
        want_off, want_place, _ = rows_of(want_idx, E)
        assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(place.cpu().numpy(), want_place)
        f = kept(T * D, drop.p, drop.seed, it, drop.site, 0).reshape(T, D)
        y64 = np.zeros((T, K, D))
        for t in range(T):
            for j in range(K):
                if want_idx[t, j] >= 0:
                    y64[t, j] = x64[t] @ w64[want_idx[t, j]]
        out64 = f64(res) + f * (wt64[..., None] * y64).sum(1)
        size = np.abs(f64(res)) + f * (wt64[..., None] * np.abs(y64)).sum(1)
        assert np.all(np.abs(f64(out) - out64) <= 3 * 2.0 ** -8 * size + 1e-6)
        d = f64(dout) * f
        dwt64 = np.einsum("td,tkd->tk", d, y64)
        gw64, dx64 = np.zeros((E, D, D)), np.zeros((T, D))
        for t in range(T):
            for j in range(K):
                e = want_idx[t, j]
                if e >= 0:
                    gw64[e] += np.outer(x64[t], wt64[t, j] * d[t])
                    dx64[t] += w64[e] @ (wt64[t, j] * d[t])
        dl64 = route_grad(l64, want_idx, dwt64, HP)
        gr64 = x64.T @ dl64
        for got, want in ((gw, gw64), (dx, dx64), (dwt, dwt64), (dlogits, dl64), (gr, gr64)):
            assert np.linalg.norm(f64(got) - want) <= 3 * 2.0 ** -8 * np.linalg.norm(want), it
        # ---- steps: the experts that no token took keep their weights' gradient at zero
        osa.optim_step_route_bias(off, bias, rate)
        loads = np.diff(want_off)
        assert np.allclose(f64(bias), b64 + 1e-2 * np.sign(loads.sum() - E * loads), atol=1e-7)
        before = [w.clone(), router.clone()]
        osa.optim_step_adamw(adam.handle, osa.optim_adamw_hp(0.9, 0.999, 1e-8), sc.lr, None, None, sc.step)
        torch.cuda.synchronize()
        assert sc.step.item() == it + 1
        assert all(bool(torch.isfinite(p).all()) and not torch.equal(p, q) for p, q in zip((w, router), before))


@pytest.mark.parametrize("tokens", [40, 5000])
def test_the_chain_in_a_graph(tokens):
    """Captured once, replayed on other inputs and steps with eager work between:
    every result is the eager call's, bit for bit.  (5000 tokens' rows go through
    the workspace.)"""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    experts, topk, dim = 32, 2, 72
    hp = osa.optim_route_hp(topk, osa.OPTIM_ROUTE_SOFTMAX, 0)
    drop = osa.optim_dropout_hp(0.3, 5, 1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    inputs = {"logits": rnd(tokens, experts), "x": rnd(tokens, dim), "dout": rnd(tokens, dim), "bias": rnd(experts) * 0.01,
              "step": torch.zeros(1, dtype=torch.int32, device=DEV)}
    rate = torch.tensor([1e-3], device=DEV)

    def fresh():
        n = osa.optim_route_rows_workspace(tokens, topk, experts)
        return {"idx": torch.zeros(tokens, topk, dtype=torch.int32, device=DEV), "w": torch.zeros(tokens, topk, device=DEV),
                "off": torch.zeros(experts + 1, dtype=torch.int32, device=DEV),
                "place": torch.zeros(tokens, topk, dtype=torch.int32, device=DEV),
                "order": torch.zeros(tokens * topk, dtype=torch.int32, device=DEV),
                "rows": torch.zeros(tokens * topk, dim, device=DEV), "out": torch.zeros(tokens, dim, device=DEV),
                "dy": torch.zeros(tokens * topk, dim, device=DEV), "dw": torch.zeros(tokens, topk, device=DEV),
                "dlogits": torch.zeros(tokens, experts, device=DEV), "bias": torch.zeros(experts, device=DEV),
                "ws": torch.empty(n, dtype=torch.uint8, device=DEV) if n else None}

    def chain(b):
        b["bias"].copy_(inputs["bias"])
        osa.optim_route(inputs["logits"], hp, b["idx"], b["w"], bias=b["bias"])
        osa.optim_route_rows(b["idx"], b["off"], b["place"], order=b["order"], workspace=b["ws"])
        osa.optim_expert_gather(inputs["x"], b["place"], b["rows"])
        osa.optim_expert_combine(b["rows"], b["place"], b["out"], weights=b["w"], residual=inputs["x"], dropout=drop, step=inputs["step"])
        osa.optim_expert_combine_grad(inputs["dout"], b["rows"], b["place"], b["dy"], weights=b["w"], dweights=b["dw"], dropout=drop,
                                      step=inputs["step"])
        osa.optim_route_grad(inputs["logits"], hp, b["idx"], b["dw"], b["dlogits"])
        osa.optim_step_route_bias(b["off"], b["bias"], rate)

    captured, eager = fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            chain(captured)
    torch.cuda.synchronize()
    for turn in range(3):
        for key in ("logits", "x", "dout"):
            inputs[key].copy_(rnd(*inputs[key].shape))
        inputs["step"].fill_(turn)
        graph.replay()
        chain(eager)
        torch.cuda.synchronize()
        for key in captured:
            if key != "ws":
                assert torch.equal(captured[key], eager[key]), (turn, key)


def test_two_layers_at_once():
    """Two layers on two streams, each with its own workspace, as one after the other."""
    sets = []
    for seed in (1, 2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        logits = torch.randn(20000, 64, generator=g, device=DEV)
        n = osa.optim_route_rows_workspace(20000, 4, 64)
        make = lambda: [torch.zeros(20000, 4, dtype=torch.int32, device=DEV), torch.zeros(20000, 4, device=DEV),  # noqa: E731
                        torch.zeros(65, dtype=torch.int32, device=DEV), torch.zeros(20000, 4, dtype=torch.int32, device=DEV),
                        torch.zeros(n, dtype=torch.uint8, device=DEV)]
        sets.append((logits, make(), make()))
    hp = osa.optim_route_hp(4)

    def run(logits, b, stream=None):
        for _ in range(5):
            osa.optim_route(logits, hp, b[0], b[1], stream=stream)
            osa.optim_route_rows(b[0], b[2], b[3], workspace=b[4], stream=stream)

    for logits, a, _ in sets:
        run(logits, a)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for (logits, _, b), s in zip(sets, streams):
        run(logits, b, s)
    torch.cuda.synchronize()
    for _, a, b in sets:
        assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
