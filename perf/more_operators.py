"""Cases and plain forms of what a mixture of experts needs around its weight gradients: routing with its gradient, the
experts' rows and the step of the balance bias, rows to the experts and back, and dropout from a counter.

``own`` false: elementary torch operations in 32 bits (64 where a choice hangs on them), rounded once at the end.  ``own``
true: this package's calls.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LARGEST = torch.finfo(torch.float32).max
BIAS_RATE = 1e-3
# Philox4x32-10 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011)
PHILOX_M, PHILOX_W, ROUNDS = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85), 10
WORD = 0xFFFFFFFF


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a reply: latency only
        {"name": "route 1x256 sigmoid groups f32", "op": "route", "tokens": 1, "experts": 256, "topk": 8, "dtype": "f32",
         "score": "sigmoid", "renormalise": True, "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "scale": 2.5, "padded": False},
        # a training batch of a layer with few experts, logits in 16 bits (many equal ones), the batch's end padded
        {"name": "route 16384x64 softmax bf16", "op": "route", "tokens": 16384, "experts": 64, "topk": 6, "dtype": "bf16",
         "score": "softmax", "renormalise": False, "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "scale": 1.0, "padded": True},
        # a large batch over many experts in groups, chosen with the balance bias
        {"name": "route 65536x256 sigmoid groups f32", "op": "route", "tokens": 65536, "experts": 256, "topk": 8, "dtype": "f32",
         "score": "sigmoid", "renormalise": True, "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "scale": 2.5, "padded": False},
        # its backward pass where the whole softmax counts
        {"name": "route grad 65536x256 softmax bf16", "op": "route grad", "tokens": 65536, "experts": 256, "topk": 8, "dtype": "bf16",
         "score": "softmax", "renormalise": False, "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "scale": 1.0, "padded": True},
        # a test model's batch: latency
        {"name": "rows 300x2 of 8", "op": "rows", "tokens": 300, "experts": 8, "topk": 2, "skew": 1.0, "padded": False},
        # a large batch, loads far from even, the end padded
        {"name": "rows 65536x8 of 256", "op": "rows", "tokens": 65536, "experts": 256, "topk": 8, "skew": 3.0, "padded": True},
        # tokens to their experts
        {"name": "gather 16384x2048 k8 bf16", "op": "gather", "tokens": 16384, "experts": 64, "topk": 8, "dim": 2048, "dtype": "bf16",
         "skew": 1.0, "padded": False, "weights": False, "residual": False, "p": 0.0},
        # one token's results back, for a reply
        {"name": "combine 1x4096 k8 bf16", "op": "combine", "tokens": 1, "experts": 256, "topk": 8, "dim": 4096, "dtype": "bf16",
         "skew": 1.0, "padded": False, "weights": True, "residual": True, "p": 0.0},
        # a training batch's results back, dropped out and added to the residual stream
        {"name": "combine 16384x4096 k2 bf16 dropout", "op": "combine", "tokens": 16384, "experts": 8, "topk": 2, "dim": 4096,
         "dtype": "bf16", "skew": 1.0, "padded": False, "weights": True, "residual": True, "p": 0.1},
        # the backward pass of a batch of odd size whose end is padded
        {"name": "combine grad 20001x1000 k4 f16 dropout", "op": "combine grad", "tokens": 20001, "experts": 64, "topk": 4, "dim": 1000,
         "dtype": "f16", "skew": 1.0, "padded": True, "weights": True, "residual": False, "p": 0.1},
        # a short odd vector: latency
        {"name": "dropout 999 f32", "op": "dropout", "numel": 999, "first": 0, "dtype": "f32", "residual": False, "p": 0.1},
        # a block's output added to the residual stream, far beyond every cache
        {"name": "dropout 134M bf16 residual", "op": "dropout", "numel": 134217728, "first": 0, "dtype": "bf16", "residual": True, "p": 0.1},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route", "route grad", "rows", "gather", "combine", "combine grad", "dropout"])
    if op == "dropout":
        return {"op": op, "numel": _log_uniform(rng, 1, 67108864), "first": rng.choice([0, 0, 5, 1 << 35]),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "residual": rng.random() < 0.5,
                "p": rng.choice([0.1, 0.5, rng.random()])}
    experts, padded = _log_uniform(rng, 4, 512), rng.random() < 0.4
    if op == "rows":
        return {"op": op, "tokens": _log_uniform(rng, 1, 65536), "experts": experts, "topk": rng.randint(1, min(experts, 8)),
                "skew": rng.choice([0.5, 1.0, 3.0]), "padded": padded}
    if op in ("route", "route grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = max(groups, 4, experts // groups * groups) if experts >= 2 * groups else experts
        groups = groups if experts % groups == 0 and experts >= 2 * groups else 1
        top_groups, bias = rng.randint((groups + 1) // 2, groups), rng.random() < 0.5
        topk = rng.randint(1, min(experts // groups * top_groups, 16))
        return {"op": op, "tokens": min(_log_uniform(rng, 1, 65536), (1 << 24) // experts), "experts": experts,
                "topk": topk, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "renormalise": topk > 1 and rng.random() < 0.5, "bias": bias,
                "groups": groups, "top_groups": top_groups, "group_best": rng.choice([1, 2]) if groups > 1 and bias else 1,
                "scale": rng.choice([1.0, 2.5]), "padded": padded}
    topk, dim = rng.randint(1, min(experts, 8)), _log_uniform(rng, 16, 8192)
    if rng.random() < 0.5:
        dim = (dim + 7) // 8 * 8
    return {"op": op, "tokens": min(_log_uniform(rng, 1, 65536), (1 << 27) // ((2 * topk + 1) * dim)), "experts": experts, "topk": topk, "dim": dim,
            "dtype": rng.choice(["f32", "bf16", "f16"]), "skew": rng.choice([0.5, 1.0, 3.0]), "padded": padded,
            "weights": op == "combine grad" or rng.random() < 0.5, "residual": op == "combine" and rng.random() < 0.5,
            "p": rng.choice([0.0, 0.1, rng.random() * 0.9]) if op != "gather" else 0.0}


def work(case):
    op, size = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "dropout":
        return {"bytes": case["numel"] * size * (3 if case["residual"] else 2), "flops": case["numel"] * 2}
    t, e, k = case["tokens"], case["experts"], case["topk"]
    if op == "route":
        return {"bytes": t * e * size + t * k * 8 + (4 * e if case["bias"] else 0), "flops": t * e * 4}
    if op == "route grad":
        whole = case["score"] == "softmax" and not case["renormalise"]
        return {"bytes": t * e * size + t * (e if whole else k) * size + t * k * 8, "flops": t * (e if whole else k) * 6}
    if op == "rows":
        return {"bytes": t * k * 12 + e * 12, "flops": t * k * 2}
    d = case["dim"]
    if op == "gather":
        return {"bytes": t * (1 + k) * d * size + t * k * (8 if case["weights"] else 4), "flops": t * k * d if case["weights"] else 0}
    if op == "combine":
        return {"bytes": t * (1 + k + case["residual"]) * d * size + t * k * (8 if case["weights"] else 4), "flops": 2 * t * k * d}
    return {"bytes": t * (1 + 2 * k) * d * size + t * k * 12, "flops": 3 * t * k * d}


# ---------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(gen, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).mul_(std).to(dtype)


def prepare(case, seed):
    return {"route": _prepare_route, "route grad": _prepare_route, "dropout": _prepare_dropout}.get(case["op"], _prepare_rows)(case, seed)


def _hp(case):
    """What the package's calls take of a routing case."""
    import optimizer_step_adamw_amd as osa
    return osa.optim_route_hp(topk=case["topk"], score={"softmax": osa.OPTIM_ROUTE_SOFTMAX, "sigmoid": osa.OPTIM_ROUTE_SIGMOID}[case["score"]],
                              renormalise=int(case["renormalise"]), groups=case["groups"], top_groups=case["top_groups"],
                              group_best=case["group_best"], scale=case["scale"])


def _prepare_route(case, seed):
    gen, t, e, k = _generator(seed), case["tokens"], case["experts"], case["topk"]
    logits = _normal(gen, (t, e), 1.5, DTYPES[case["dtype"]])
    if case["padded"]:  # rows behind the batch's end: no expert is open to them
        logits[t - t // 10:] = -math.inf
    spread = 0.3 if case["score"] == "sigmoid" else 2.0 / e
    s = {"case": case, "logits": logits, "bias": _normal(gen, (e,), 0.2 * spread) if case["bias"] else None,
         "idx": torch.empty(t, k, dtype=torch.int32, device=DEV), "weights": torch.empty(t, k, device=DEV)}
    if own:
        s["hp"] = _hp(case)
    if case["op"] == "route grad":
        s["idx"].copy_(_choose(case, logits, s["bias"]))
        s["dweights"] = _normal(gen, (t, k), 1e-2)
        s["dlogits"] = torch.empty_like(logits)
    return s


def _prepare_rows(case, seed):
    gen, t, e, k = _generator(seed), case["tokens"], case["experts"], case["topk"]
    # each token's experts drawn without putting back, some far likelier than others
    liking = torch.rand(e, generator=gen, device=DEV).pow(case["skew"]).add_(1e-3).log()
    noise = torch.rand(t, e, generator=gen, device=DEV).clamp_(1e-7, 1 - 1e-7)
    idx = (liking - (-noise.log()).log()).topk(k).indices.to(torch.int32)
    if case["padded"]:  # rows behind the batch's end go nowhere, and here and there a choice was dropped
        idx[torch.rand(t, k, generator=gen, device=DEV) < 0.02] = -1
        idx[t - t // 10:] = -1
    s = {"case": case, "idx": idx, "offsets": torch.empty(e + 1, dtype=torch.int32, device=DEV),
         "order": torch.empty(t * k, dtype=torch.int32, device=DEV), "place": torch.empty(t, k, dtype=torch.int32, device=DEV)}
    if case["op"] == "rows":
        s["bias"], s["rate"] = _normal(gen, (e,), 0.05), torch.tensor([BIAS_RATE], device=DEV)
        if own:
            import optimizer_step_adamw_amd as osa
            nbytes = osa.optim_route_rows_workspace(t, k, e)
            s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
        return s
    s["offsets"], s["order"], s["place"] = _rows(idx, e)
    dt, d = DTYPES[case["dtype"]], case["dim"]
    weights = torch.rand(t, k, generator=gen, device=DEV)
    s["weights"] = weights / weights.sum(1, keepdim=True) if case["weights"] else None
    s["tokens"] = _normal(gen, (t, d), 1.0, dt)  # the experts' input, or the gradient of what they gave
    s["rows"] = _normal(gen, (t * k, d), 1.0, dt)
    s["residual"] = _normal(gen, (t, d), 1.0, dt) if case["residual"] else None
    s["out"] = torch.zeros(t * k if case["op"] != "combine" else t, d, dtype=dt, device=DEV)
    s["dweights"] = torch.zeros(t, k, device=DEV)
    _prepare_draws(s, case, gen)
    return s


def _prepare_dropout(case, seed):
    gen, n, dt = _generator(seed), case["numel"], DTYPES[case["dtype"]]
    s = {"case": case, "x": _normal(gen, (n,), 1.0, dt), "residual": _normal(gen, (n,), 1.0, dt) if case["residual"] else None,
         "out": torch.empty(n, dtype=dt, device=DEV)}
    _prepare_draws(s, case, gen)
    return s


def _prepare_draws(s, case, gen):
    """What a mask is drawn from: the program's seed, the layer's number and the step that the device counts."""
    s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=gen, device=DEV))
    s["site"], s["first"] = 3, case.get("first", 0)
    s["step"] = torch.randint(0, 100000, (1,), generator=gen, device=DEV, dtype=torch.int32)
    if own and case["p"]:
        import optimizer_step_adamw_amd as osa
        s["drop"] = osa.optim_dropout_hp(p=case["p"], seed=s["seed"], site=s["site"], first=s["first"])


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"route": _run_route, "route grad": _run_route_grad, "rows": _run_rows, "gather": _run_gather, "combine": _run_combine,
            "combine grad": _run_combine_grad, "dropout": _run_dropout}[state["case"]["op"]](state)


def _logits(logits):
    """As floats: +inf is the largest one, and what no expert may have is -inf."""
    return logits.float().nan_to_num(nan=-math.inf, posinf=LARGEST, neginf=-math.inf)


def _scores(case, l):
    """Scores of finite or -inf logits, in the logits' type; zero in a row that has none."""
    if case["score"] == "sigmoid":
        return 1 / (1 + (-l).exp())
    most = l.amax(1, keepdim=True).clamp(min=-LARGEST)
    p = (l - most).exp()
    return p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _choose(case, logits, bias):
    """The chosen experts, -1 where none is left: by scores and bias in 64 bits, or by the logits, which order the scores."""
    l, t = _logits(logits), logits.shape[0]
    c = l.double()
    if bias is not None or case["group_best"] > 1:
        c = _scores(case, c)
        c = torch.where(l > -math.inf, c if bias is None else c + bias.double(), -math.inf)
    if case["groups"] > 1:
        g = c.view(t, case["groups"], -1)
        best = g.sort(dim=2, descending=True).values[:, :, :case["group_best"]]
        rank = torch.where(best[:, :, 0] > -math.inf, torch.where(best > -math.inf, best, 0.0).sum(2), -math.inf)
        kept = rank.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros_like(rank).scatter_(1, kept, 1.0) > 0
        c = torch.where(open_[:, :, None], g, -math.inf).view(t, -1)
    best = c.sort(dim=1, descending=True, stable=True)
    return torch.where(best.values > -math.inf, best.indices, -1)[:, :case["topk"]].to(torch.int32)


def _run_route(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_route(s["logits"], s["hp"], s["idx"], s["weights"], bias=s["bias"])
        return {"idx": s["idx"], "weights": s["weights"]}
    case = s["case"]
    idx = _choose(case, s["logits"], s["bias"])
    w = _scores(case, _logits(s["logits"])).gather(1, idx.long().clamp(min=0)) * (idx >= 0)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    return {"idx": idx, "weights": w * case["scale"] + 0 * s["logits"].isnan().any(1, keepdim=True)}


def _run_route_grad(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_route_grad(s["logits"], s["hp"], s["idx"], s["dweights"], s["dlogits"])
        return s["dlogits"]
    case, scores = s["case"], _scores(s["case"], _logits(s["logits"]))
    chosen, at = s["idx"] >= 0, s["idx"].long().clamp(min=0)
    g = torch.where(chosen, s["dweights"], 0.0) * case["scale"]
    sc = scores.gather(1, at) * chosen
    if case["renormalise"]:
        total = sc.sum(1, keepdim=True).clamp(min=1e-30)
        g = chosen * (g - (g * sc / total).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(scores).scatter_add_(1, at, g)
    if case["score"] == "sigmoid":
        dl = ds * scores * (1 - scores)
    else:
        dl = scores * (ds - (scores * ds).sum(1, keepdim=True))
    s["dlogits"].copy_(dl)
    return s["dlogits"]


def _rows(idx, experts):
    """First row of each expert's run and the end, the choice that each row holds, and the row of each choice."""
    none = idx.flatten() < 0
    by = torch.where(none, experts, idx.flatten())
    values, order = by.sort(stable=True)
    offsets = torch.searchsorted(values, torch.arange(experts + 1, device=DEV, dtype=torch.int32))
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=DEV))
    return (offsets.to(torch.int32), torch.where(values < experts, order, -1).to(torch.int32),
            torch.where(none, -1, place).to(torch.int32).view(idx.shape))


def _run_rows(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_route_rows(s["idx"], s["offsets"], s["place"], order=s["order"], workspace=s["workspace"])
        osa.optim_step_route_bias(s["offsets"], s["bias"], s["rate"])
        return {"offsets": s["offsets"], "order": s["order"], "place": s["place"], "bias": s["bias"]}
    experts = s["case"]["experts"]
    offsets, order, place = _rows(s["idx"], experts)
    load = offsets.diff().long()
    s["bias"].add_(s["rate"] * (load.sum() - experts * load).sign())
    return {"offsets": offsets, "order": order, "place": place, "bias": s["bias"]}


def _philox(block, step, site, seed):
    """Four random words of 32 bits for every counter (block, step, site)."""
    def one(state, r):
        a, b, c, d = state
        x, y = a * PHILOX_M[0], c * PHILOX_M[1]  # the low 64 bits of the products, as whole numbers with a sign
        k0, k1 = ((seed & WORD) + r * PHILOX_W[0]) & WORD, ((seed >> 32) + r * PHILOX_W[1]) & WORD
        return ((y >> 32) & WORD) ^ b ^ k0, y & WORD, ((x >> 32) & WORD) ^ d ^ k1, x & WORD

    begin = (block & WORD, block >> 32, torch.zeros_like(block) + step.long(), torch.full_like(block, site))
    return functools.reduce(one, range(ROUNDS), begin)


def _drop(s, x):
    """Floats `x`, their flat places counted from the state's first one, each dropped or scaled."""
    p = s["case"]["p"]
    if not p:
        return x
    bar, n, first = min(65535, round(p * 65536)), x.numel(), s["first"]
    block = torch.arange(first >> 3, (first + n + 7) >> 3, device=DEV)
    words = torch.stack(_philox(block, s["step"], s["site"], s["seed"]), 1)
    draws = torch.stack([words & 0xFFFF, words >> 16], 2).flatten()[first & 7:][:n].view(x.shape)
    return torch.where(draws >= bar, x * (65536 / (65536 - bar)), 0.0)


def _run_gather(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_expert_gather(s["tokens"], s["place"], s["out"], weights=s["weights"])
        return s["out"]
    order = s["order"].long()
    x = s["tokens"].float()[order.clamp(min=0) // s["case"]["topk"]]
    if s["weights"] is not None:
        x = x * s["weights"].flatten()[order.clamp(min=0)][:, None]
    s["out"].copy_(torch.where(order[:, None] >= 0, x, s["out"].float()))
    return s["out"]


def _chosen_rows(s):
    """The rows of each token's choices, zeros where there is none."""
    place = s["place"].long()
    return torch.where(place[..., None] >= 0, s["rows"].float()[place.clamp(min=0)], 0.0)


def _run_combine(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_expert_combine(s["rows"], s["place"], s["out"], weights=s["weights"], residual=s["residual"], dropout=s.get("drop"),
                                 step=s["step"])
        return s["out"]
    y = _chosen_rows(s)
    out = _drop(s, (y if s["weights"] is None else y * s["weights"][..., None]).sum(1))
    s["out"].copy_(out if s["residual"] is None else s["residual"].float() + out)
    return s["out"]


def _run_combine_grad(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_expert_combine_grad(s["tokens"], s["rows"], s["place"], s["out"], weights=s["weights"], dweights=s["dweights"],
                                      dropout=s.get("drop"), step=s["step"])
        return {"dy": s["out"], "dweights": s["dweights"]}
    d, order = _drop(s, s["tokens"].float()), s["order"].long()
    at = order.clamp(min=0)
    dy = d[at // s["case"]["topk"]] * s["weights"].flatten()[at][:, None]
    s["out"].copy_(torch.where(order[:, None] >= 0, dy, s["out"].float()))
    s["dweights"].copy_((_chosen_rows(s) * d[:, None, :]).sum(2))
    return {"dy": s["out"], "dweights": s["dweights"]}


def _run_dropout(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_dropout(s["x"], s["out"], s["drop"], residual=s["residual"], step=s["step"])
        return s["out"]
    y = _drop(s, s["x"].float())
    s["out"].copy_(y if s["residual"] is None else s["residual"].float() + y)
    return s["out"]


# ---------------------------------------------------------------------------------------------- in 64 bits
def _kept(s, shape):
    """Share of itself that each element keeps (0, or 1 over the share kept), the generator's products by halves of words."""
    p, n, first = s["case"]["p"], math.prod(shape), s["first"]
    if not p:
        return torch.ones(shape, dtype=torch.float64, device=DEV)
    bar, low = min(65535, int(p * 65536 + 0.5)), 0xFFFF

    def product(a, m):  # (high, low) word
        mid = (a >> 16) * (m & low) + ((a & low) * (m & low) >> 16)
        mid2 = (a & low) * (m >> 16) + (mid & low)
        return (a >> 16) * (m >> 16) + (mid >> 16) + (mid2 >> 16), (mid2 & low) << 16 | (a & low) * (m & low) & low

    c = [torch.arange(first // 8, (first + n - 1) // 8 + 1, device=DEV)]
    c = [c[0] % 2 ** 32, c[0] // 2 ** 32, int(s["step"]) + 0 * c[0], s["site"] + 0 * c[0]]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for _ in range(ROUNDS):
        (h0, l0), (h1, l1) = product(c[0], PHILOX_M[0]), product(c[2], PHILOX_M[1])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[i] + PHILOX_W[i]) % 2 ** 32 for i in (0, 1)]
    draws = torch.empty(c[0].numel(), 8, dtype=torch.int32, device=DEV)
    for i in range(4):
        draws[:, 2 * i] = (c[i] % 65536).to(torch.int32)
        draws[:, 2 * i + 1] = (c[i] // 65536).to(torch.int32)
    draws = draws.view(-1)[first % 8:first % 8 + n]
    return (draws >= bar).double().mul_(65536.0 / (65536 - bar)).view(shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        y = s["x"].double() * _kept(s, s["x"].shape)
        return y if s["residual"] is None else y + s["residual"].double()
    if op in ("route", "route grad"):
        return _exact_route(case, s)
    if op == "rows":
        load = torch.stack([(s["idx"] == e).sum() for e in range(case["experts"])])
        even = load.sum().double() / case["experts"]
        return {"offsets": None, "order": None, "place": None, "bias": s["bias"].double() + float(s["rate"]) * torch.sign(even - load)}
    place, rows = s["place"].long(), s["rows"].double()
    w = s["weights"].double() if s["weights"] is not None else torch.ones(place.shape, dtype=torch.float64, device=DEV)
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            of = (place[:, j] >= 0).nonzero().flatten()
            out[of] += rows[place[of, j]] * w[of, j, None]
        out = out * _kept(s, out.shape)
        return out if s["residual"] is None else out + s["residual"].double()
    x = s["tokens"].double()
    if op == "combine grad":
        x = x * _kept(s, x.shape)
    out, dw = s["out"].double(), torch.zeros(place.shape, dtype=torch.float64, device=DEV)
    for j in range(case["topk"]):
        of = (place[:, j] >= 0).nonzero().flatten()
        out[place[of, j]] = x[of] * w[of, j, None]
        if op == "combine grad":
            dw[of, j] = (x[of] * rows[place[of, j]]).sum(1)
    return out if op == "gather" else {"dy": out, "dweights": dw}


def _exact_route(case, s):
    """Row by row in the order of the definition, all rows at a time: the best one left is taken, topk times."""
    l = s["logits"].double()
    if case["score"] == "softmax":
        scores = torch.softmax(l, 1).nan_to_num(0.0)
    else:
        scores = torch.sigmoid(l)
    if case["op"] == "route grad":
        # the weights' derivative by every score, then the scores' by every logit
        chosen = torch.zeros_like(l, dtype=torch.bool)
        g = torch.zeros_like(l)
        for j in range(case["topk"]):
            of = (s["idx"][:, j] >= 0).nonzero().flatten()
            chosen[of, s["idx"][of, j].long()] = True
            g[of, s["idx"][of, j].long()] = s["dweights"][of, j].double() * case["scale"]
        if case["renormalise"]:
            total = (scores * chosen).sum(1, keepdim=True)
            total = torch.where(total > 0, total, 1.0)
            g = torch.where(chosen, g / total - (g * scores).sum(1, keepdim=True) / total ** 2, 0.0)
        if case["score"] == "sigmoid":
            return g * scores * (1 - scores)
        return scores * g - scores * (scores * g).sum(1, keepdim=True)
    c = scores if s["bias"] is None else scores + s["bias"].double()
    c = torch.where(l == -math.inf, -math.inf, c)
    if case["groups"] > 1:
        per = case["experts"] // case["groups"]
        best = torch.stack([c[:, i * per:(i + 1) * per].topk(min(case["group_best"], per)).values for i in range(case["groups"])], 1)
        rank = torch.where(best[:, :, 0].isinf(), -math.inf, best.masked_fill(best.isinf(), 0.0).sum(2))
        for _ in range(case["groups"] - case["top_groups"]):  # the worst group left is shut, the later one of equals
            worst = case["groups"] - 1 - rank.flip(1).min(1).indices
            shut = torch.arange(case["experts"], device=DEV)[None] // per == worst[:, None]
            c = torch.where(shut, -math.inf, c)
            rank.scatter_(1, worst[:, None], math.inf)
    w = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    left = c.clone()
    for j in range(case["topk"]):
        best = left.max(1)
        w[:, j] = torch.where(best.values > -math.inf, scores.gather(1, best.indices[:, None])[:, 0], 0.0)
        left.scatter_(1, best.indices[:, None], -math.inf)
    if case["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"idx": None, "weights": w * case["scale"]}
