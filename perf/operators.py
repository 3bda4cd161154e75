"""Cases and plain forms of the operators around an optimizer step: norms of many gradients and clipping in place, the
weight gradients of a mixture of experts, and the Muon step of a list of matrices.

``own`` false: elementary torch operations in 32 bits, rounded once at the end.  ``own`` true: this package's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# loss scale of 16-bit gradients (a training loop that unscales with the clip)
LOSS_SCALE = 65536.0
# quintic of the orthogonalisation (K. Jordan et al., "Muon: An optimizer for hidden layers in neural networks", 2024)
NS_A, NS_B, NS_C, NS_STEPS = 3.4445, -4.7750, 2.0315, 5
MUON_MOMENTUM, MUON_EPS, MUON_LR, MUON_WD = 0.95, 1e-7, 0.02, 0.1


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # logging every tensor's norm of a 1.1B-parameter list, 16-bit gradients under a loss scale
        {"name": "norms list 1.1B bf16", "op": "norms", "dtype": "bf16", "kind": "l2", "lists": "llama", "layers": 16,
         "dim": 2048, "ffn": 8192, "vocab": 32000},
        # thousands of bias and norm vectors: launches and tables, not bytes
        {"name": "norms 6000 vectors f32", "op": "norms", "dtype": "f32", "kind": "l2", "lists": "ragged", "count": 6000,
         "low": 1, "high": 700},
        # a two-layer test model: latency only
        {"name": "clip tiny model f32", "op": "clip", "dtype": "f32", "kind": "l2", "lists": "llama", "layers": 2,
         "dim": 64, "ffn": 172, "vocab": 256},
        # one matrix whose gradient fits the last-level cache
        {"name": "clip 4096x4096 f32", "op": "clip", "dtype": "f32", "kind": "l2", "lists": "ragged", "count": 1,
         "low": 16777216, "high": 16777216},
        # embeddings and two layers of a 7B list: far beyond every cache
        {"name": "clip list 667M bf16", "op": "clip", "dtype": "bf16", "kind": "l2", "lists": "llama", "layers": 2,
         "dim": 4096, "ffn": 11008, "vocab": 32000},
        # a bucket of odd-sized tensors, none of them aligned, clipped by the largest magnitude
        {"name": "clip ragged bucket f16", "op": "clip", "dtype": "f16", "kind": "inf", "lists": "ragged", "count": 300,
         "low": 1000, "high": 1000000},
        # a test model's experts with a handful of tokens each: latency
        {"name": "expert 4x256x172 f16", "op": "expert", "dtype": "f16", "out": "f32", "experts": 4, "m": 256, "n": 172,
         "tokens": 300, "skew": 1.0, "accumulate": True},
        # a micro-batch accumulated into fp32 gradients, few wide experts
        {"name": "expert 8x2048x8192 bf16", "op": "expert", "dtype": "bf16", "out": "f32", "experts": 8, "m": 2048,
         "n": 8192, "tokens": 16384, "skew": 1.0, "accumulate": True},
        # many narrow experts, some with most of the tokens and some with none, gradients kept in 16 bits
        {"name": "expert 64x2048x1024 bf16", "op": "expert", "dtype": "bf16", "out": "bf16", "experts": 64, "m": 2048,
         "n": 1024, "tokens": 65536, "skew": 3.0, "accumulate": False},
        # the two-layer test model's matrices: latency
        {"name": "muon tiny model f32", "op": "muon", "param": "f32", "grad": "f32", "copies": 2,
         "shapes": "4x64x64,2x172x64,1x64x172", "nesterov": True},
        # experts' weights stacked in one tensor, odd sizes, a bf16 model copy beside fp32 masters
        {"name": "muon 24 experts 1000x408", "op": "muon", "param": "bf16", "grad": "bf16", "copies": 2,
         "shapes": "24x1000x408", "nesterov": True},
        # the matrices of one layer of a 7B list
        {"name": "muon layer d4096 f32", "op": "muon", "param": "f32", "grad": "f32", "copies": 1,
         "shapes": "4x4096x4096,2x11008x4096,1x4096x11008", "nesterov": True},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norms", "clip", "expert", "muon"])
    if op in ("norms", "clip"):
        high = _log_uniform(rng, 64, 8_000_000)
        count = max(1, min(_log_uniform(rng, 1, 6000), 200_000_000 // high))
        return {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "kind": rng.choice(["l2", "l2", "inf", "l1"]),
                "lists": "ragged", "count": count, "low": max(1, high // rng.choice([1, 10, 1000])), "high": high}
    if op == "expert":
        m, n = _log_uniform(rng, 64, 4096), _log_uniform(rng, 64, 4096)
        experts = min(_log_uniform(rng, 1, 64), (1 << 27) // (m * n))
        if rng.random() < 0.6:
            m, n = (m + 7) // 8 * 8, (n + 7) // 8 * 8
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "out": rng.choice(["f32", "bf16"]), "experts": experts,
                "m": m, "n": n, "tokens": _log_uniform(rng, 1, 32768), "skew": rng.choice([0.5, 1.0, 3.0]),
                "accumulate": rng.random() < 0.5}
    groups = []
    for _ in range(rng.randint(1, 3)):
        r, c = _log_uniform(rng, 16, 4096), _log_uniform(rng, 16, 4096)
        count = max(1, min(_log_uniform(rng, 1, 32), 30_000_000 // (r * c)))
        groups.append("%dx%dx%d" % (count, r, c))
    return {"op": op, "param": rng.choice(["f32", "bf16"]), "grad": rng.choice(["f32", "bf16"]),
            "copies": 1, "shapes": ",".join(groups), "nesterov": rng.random() < 0.7}


def _sizes(case):
    if case["lists"] == "llama":
        from synth import llama_list
        return [t.numel for t in llama_list(case["layers"], case["dim"], case["ffn"], case["vocab"], tied=True)]
    rng = random.Random("%(count)d %(low)d %(high)d" % case)
    return [_log_uniform(rng, case["low"], case["high"]) for _ in range(case["count"])]


def _shapes(case):
    """(matrices, rows, cols) of each tensor of the list."""
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")] * case["copies"]


def _offsets(case):
    """First row of each expert's run, and the end: shares drawn with the case's skew, some runs empty where it is high."""
    rng = random.Random("%(experts)d %(tokens)d %(skew)f" % case)
    w = [rng.random() ** case["skew"] for _ in range(case["experts"])]
    if case["skew"] > 2:
        w = [0.0 if k % 8 == 5 else v for k, v in enumerate(w)]
    total, at, out = sum(w) or 1.0, 0.0, [0]
    for v in w:
        at += v
        out.append(min(case["tokens"], int(round(case["tokens"] * at / total))))
    return out


def work(case):
    op = case["op"]
    if op in ("norms", "clip"):
        n, b = sum(_sizes(case)), 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * b * (2 if op == "clip" else 1), "flops": n * (3 if op == "clip" else 2)}
    if op == "expert":
        e, m, n, t = case["experts"], case["m"], case["n"], _offsets(case)[-1]
        out = e * m * n * (4 if case["out"] == "f32" else 2)
        return {"bytes": 2 * t * (m + n) + out * (2 if case["accumulate"] else 1), "flops": 2.0 * t * m * n}
    flops, elements = 0.0, 0
    for k, r, c in _shapes(case):
        s, g = min(r, c), max(r, c)
        flops += k * NS_STEPS * (3.0 * s * s * g + float(s) ** 3)
        elements += k * r * c
    # parameter and momentum read and written, gradient read, model copy written
    return {"bytes": elements * (16 + (4 if case["grad"] == "f32" else 2) + (2 if case["param"] == "bf16" else 0)), "flops": flops}


# ---------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _normal(gen, n, std, dtype):
    return torch.randn(n, generator=gen, device=DEV).mul_(std).to(dtype)


def _scalar(v, dtype=torch.float32):
    return torch.tensor([v], dtype=dtype, device=DEV)


def prepare(case, seed):
    return {"norms": _prepare_grads, "clip": _prepare_grads, "expert": _prepare_expert, "muon": _prepare_muon}[case["op"]](case, seed)


def _prepare_grads(case, seed):
    gen, sizes = _generator(seed), _sizes(case)
    scale = 1.0 if case["dtype"] == "f32" else LOSS_SCALE
    # every gradient lies in one bucket, end to end, as data-parallel training keeps them
    flat = _normal(gen, sum(sizes), 1e-3 * scale, DTYPES[case["dtype"]])
    grads = list(flat.split(sizes))
    s = {"op": case["op"], "kind": case["kind"], "flat": flat, "grads": grads, "sizes": sizes, "inv_scale": _scalar(1.0 / scale)}
    # the bar lies at about half the norm
    whole = {"l2": 1e-3 * math.sqrt(sum(sizes)), "l1": 1e-3 * 0.8 * sum(sizes), "inf": 1e-3 * math.sqrt(2 * math.log(sum(sizes) + 1))}
    s["max_norm"] = 0.5 * whole[case["kind"]]
    if len(sizes) > 64 and sum(sizes) < 1 << 26:  # many and small: where each begins and ends, for running sums
        s["ends"] = torch.tensor(sizes, device=DEV).cumsum(0)
    s["found_inf"], s["one"] = _scalar(0.0), _scalar(1.0)
    s["norms"], s["total"], s["coef"] = torch.zeros(len(sizes), device=DEV), _scalar(0.0), _scalar(0.0)
    if own:
        import optimizer_step_adamw_amd as osa
        s["plan"] = osa.Plan(osa.grad_list(grads), osa.OPTIM_ALGO_GRADS)
    return s


def _prepare_expert(case, seed):
    gen, off = _generator(seed), _offsets(case)
    e, m, n, t = case["experts"], case["m"], case["n"], case["tokens"]
    dt = DTYPES[case["dtype"]]
    s = {"op": "expert", "accumulate": case["accumulate"], "runs": list(zip(off, off[1:])),
         "offsets": torch.tensor(off, dtype=torch.int32, device=DEV),
         "x": _normal(gen, t * m, 1.0, dt).view(t, m), "dy": _normal(gen, t * n, 1e-2, dt).view(t, n),
         "dw": _normal(gen, e * m * n, 1e-2, DTYPES[case["out"]]).view(e, m, n)}
    if own:
        import optimizer_step_adamw_amd as osa
        nbytes = osa.optim_expert_grad_workspace(e, t, m, n)
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return s


def _prepare_muon(case, seed):
    gen, shapes = _generator(seed), _shapes(case)
    elements = [k * r * c for k, r, c in shapes]
    # gradients with a few strong directions above noise, as those of matrices have
    grads, masters, moms = [], [], []
    for k, r, c in shapes:
        u, v = torch.randn(k, r, 2, generator=gen, device=DEV), torch.randn(k, 2, c, generator=gen, device=DEV)
        noise = torch.randn(k, r, c, generator=gen, device=DEV)
        grads.append((noise + 0.5 * u @ v).mul_(1e-3).to(DTYPES[case["grad"]]))
        moms.append(torch.randn(k, r, c, generator=gen, device=DEV).mul_(5e-3))
        masters.append(torch.randn(k, r, c, generator=gen, device=DEV).mul_(0.02))
    s = {"op": "muon", "shapes": shapes, "grads": grads, "moms": moms, "masters": masters, "nesterov": case["nesterov"],
         "copies": [p.to(torch.bfloat16) for p in masters] if case["param"] == "bf16" else None,
         "lr": _scalar(MUON_LR), "step": _scalar(0, torch.int32), "lr_host": MUON_LR, "numel": elements}
    if own:
        import optimizer_step_adamw_amd as osa
        code = {"f32": osa.OPTIM_F32, "bf16": osa.OPTIM_BF16}
        tl = osa.TensorList(s["copies"] or masters, grads, m=moms, master=masters if s["copies"] else None,
                            weight_decay=[MUON_WD] * len(shapes), rows=[r for _, r, _ in shapes], cols=[c for _, _, c in shapes],
                            param_dtype=code[case["param"]], grad_dtype=code[case["grad"]])
        s["plan"] = osa.Plan(tl, osa.OPTIM_ALGO_MUON)
        s["hp"] = osa.optim_muon_hp(momentum=MUON_MOMENTUM, eps=MUON_EPS, nesterov=int(case["nesterov"]), scale_kind=osa.OPTIM_MUON_SCALE_RMS)
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"norms": _run_grads, "clip": _run_grads, "expert": _run_expert, "muon": _run_muon}[state["op"]](state)


def _run_grads(s):
    if own:
        import optimizer_step_adamw_amd as osa
        kind = {"l2": osa.OPTIM_NORM_L2, "l1": osa.OPTIM_NORM_L1, "inf": osa.OPTIM_NORM_INF}[s["kind"]]
        osa.optim_grad_norms(s["plan"].handle, kind, s["inv_scale"], s["max_norm"], s["found_inf"], s["norms"], s["total"], s["coef"])
        if s["op"] == "clip":
            osa.optim_clip_grads(s["plan"].handle, s["coef"], s["found_inf"])
        norms, total, coef = s["norms"], s["total"], s["coef"]
    else:
        x = s["flat"].float()
        y = x.abs() if s["kind"] != "l2" else x * x
        if "ends" in s and s["kind"] != "inf":
            sums = y.cumsum(0, dtype=torch.float64)[s["ends"] - 1]
            norms = torch.cat([sums[:1], sums.diff()]).float()
        else:
            norms = torch.stack([v.amax() if s["kind"] == "inf" else v.sum() for v in y.split(s["sizes"])])
        norms = (norms.sqrt() if s["kind"] == "l2" else norms) * s["inv_scale"]
        total = {"l2": lambda: norms.square().sum().sqrt(), "l1": norms.sum, "inf": norms.amax}[s["kind"]]().reshape(1)
        coef = s["inv_scale"] * (s["max_norm"] / (total + 1e-6)).clamp(max=1.0)
        s["found_inf"].copy_(torch.maximum(s["found_inf"], (~torch.isfinite(total)).float()))
        if s["op"] == "clip":
            s["flat"].copy_(x * coef)
    if s["op"] == "norms":
        return {"norms": norms, "total": total, "coef": coef, "found_inf": s["found_inf"]}
    # the clipped gradients now lie at the bar, unscaled: a pass more on them meets a slightly lower bar, as a pass on new
    # gradients would meet one that they exceed
    s["max_norm"] *= 0.99999
    s["inv_scale"] = s["one"]
    return {"norms": norms, "total": total, "coef": coef, "grads": s["flat"]}


def _run_expert(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_expert_grad(s["x"], s["dy"], s["offsets"], s["dw"], accumulate=s["accumulate"], workspace=s["workspace"])
    else:
        x, dy = s["x"].float(), s["dy"].float()
        dw = torch.stack([x[a:b].t() @ dy[a:b] for a, b in s["runs"]])
        s["dw"].copy_(s["dw"].float() + dw if s["accumulate"] else dw)
    return s["dw"]


def _orthogonal(u):
    """The direction of each matrix of the stack `u`: its singular values brought near one by five steps of the quintic."""
    x = u / (u.square().sum((1, 2), keepdim=True).sqrt() + MUON_EPS)
    wide = x.shape[1] <= x.shape[2]
    x = x if wide else x.transpose(1, 2).contiguous()
    for _ in range(NS_STEPS):
        a = x @ x.transpose(1, 2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x if wide else x.transpose(1, 2)


def _run_muon(s):
    if own:
        import optimizer_step_adamw_amd as osa
        osa.optim_step_muon(s["plan"].handle, s["hp"], s["lr"], None, None, s["step"])
    else:
        for i, (m, g, p) in enumerate(zip(s["moms"], s["grads"], s["masters"])):
            g = g.float()
            m.copy_(MUON_MOMENTUM * m + g)
            o = _orthogonal(g + MUON_MOMENTUM * m if s["nesterov"] else m)
            p.copy_(p - (s["lr"] * MUON_WD * p + s["lr"] * (0.2 * math.sqrt(max(p.shape[1:]))) * o))
            if s["copies"]:
                s["copies"][i].copy_(p)
        s["step"] += 1
    return {"masters": s["masters"], "moms": s["moms"], "copies": s["copies"] or [], "step": s["step"]}


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norms", "clip"):
        g = s["flat"].double().split(s["sizes"])
        of = {"l2": torch.linalg.vector_norm, "l1": lambda v: v.abs().sum(), "inf": lambda v: v.abs().max()}[case["kind"]]
        inv = s["inv_scale"].double()
        norms = torch.stack([of(v) for v in g]) * inv
        total = of(norms).reshape(1)
        coef = inv * min(1.0, s["max_norm"] / (float(total) + 1e-6))
        if case["op"] == "norms":
            return {"norms": norms, "total": total, "coef": coef, "found_inf": None}
        return {"norms": norms, "total": total, "coef": coef, "grads": s["flat"].double() * coef}
    if case["op"] == "expert":
        dw = s["dw"].double() if case["accumulate"] else torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(s["runs"]):
            if b > a:
                dw[e].addmm_(s["x"][a:b].double().t().contiguous(), s["dy"][a:b].double())
        return dw
    out = {"masters": [], "moms": [], "copies": [], "step": None}
    for p, g, m in zip(s["masters"], s["grads"], s["moms"]):
        g, p = g.double(), p.double()
        m = m.double() * MUON_MOMENTUM + g
        x = m * MUON_MOMENTUM + g if case["nesterov"] else m
        x = x / (torch.linalg.matrix_norm(x, keepdim=True) + MUON_EPS)
        if x.shape[1] > x.shape[2]:  # the iteration commutes with transposition: products on the shorter side
            for _ in range(NS_STEPS):
                q = torch.bmm(x.transpose(1, 2).contiguous(), x)
                x = NS_A * x + torch.bmm(x, NS_B * q + NS_C * torch.bmm(q, q))
        else:
            for _ in range(NS_STEPS):
                q = torch.bmm(x, x.transpose(1, 2).contiguous())
                x = NS_A * x + torch.bmm(NS_B * q + NS_C * torch.bmm(q, q), x)
        p = p - MUON_LR * (MUON_WD * p + 0.2 * math.sqrt(max(x.shape[1:])) * x)
        out["masters"].append(p)
        out["moms"].append(m)
        if case["param"] == "bf16":
            out["copies"].append(p)
    return out
