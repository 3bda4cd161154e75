"""Plain forms in 64 bits (numpy, on the host) of routing, the experts' rows and
dropout, written from the definitions in include/optim_route.h and
include/optim_dropout.h; a token at a time."""
from __future__ import annotations

import math

import numpy as np
import torch

import optimizer_step_adamw_amd as osa

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LARGEST = float(np.finfo(np.float32).max)


def f64(t):
    return t.detach().double().cpu().numpy()


def scores(row, score):
    """Scores of a row whose NaN and -inf are no scores at all (0)."""
    l = np.where(np.isnan(row), -np.inf, np.minimum(row, LARGEST))
    if score == osa.OPTIM_ROUTE_SIGMOID:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    if not (l > -np.inf).any():
        return np.zeros_like(l)
    e = np.exp(l - l.max())
    return e / e.sum()


def choose(row, bias, hp):
    """The chosen experts of a row, fewer than topk where no more are open."""
    n = row.size
    l = np.where(np.isnan(row), -np.inf, np.minimum(row, LARGEST))
    c = l.copy()
    if bias is not None or (hp.groups > 1 and hp.group_best > 1):
        b = np.zeros(n) if bias is None else np.where(np.isnan(bias), -np.inf, bias)
        c = np.where((l > -np.inf) & (b > -np.inf), scores(row, hp.score) + b, -np.inf)
    if hp.groups > 1:
        per = n // hp.groups
        rank = []
        for g in range(hp.groups):
            best = sorted((x for x in c[g * per:(g + 1) * per] if x > -math.inf), reverse=True)[:hp.group_best]
            rank.append(sum(best) if best else -math.inf)
        kept = sorted(range(hp.groups), key=lambda g: (-rank[g], g))[:hp.top_groups]
        c = np.where([e // per in kept for e in range(n)], c, -np.inf)
    return [e for e in sorted(range(n), key=lambda e: (-c[e], e))[:hp.topk] if c[e] > -math.inf]


def weights_of(row, idx, hp):
    """The weights of the chosen experts of a row."""
    l = np.minimum(row[idx], LARGEST) if len(idx) else np.zeros(0)
    if hp.renormalise and len(idx):
        # of the scores' logarithms, so that none vanishes
        logs = l if hp.score == osa.OPTIM_ROUTE_SOFTMAX else np.array([-np.logaddexp(0.0, -x) for x in l])
        s = np.exp(logs - logs.max())
        s = s / s.sum()
    else:
        s = scores(row, hp.score)[idx] if len(idx) else np.zeros(0)
    w = hp.scale * s
    return np.full(len(idx), np.nan) if np.isnan(row).any() else w


def route(logits, bias, hp):
    """(idx, weights) of every token, -1 and 0 behind the last choice."""
    idx = np.full((logits.shape[0], hp.topk), -1, np.int32)
    w = np.zeros((logits.shape[0], hp.topk))
    for t, row in enumerate(logits):
        at = choose(row, bias, hp)
        idx[t, :len(at)] = at
        w[t, :len(at)] = weights_of(row, at, hp)
        if np.isnan(row).any():
            w[t] = np.nan
    return idx, w


def route_grad(logits, idx, dweights, hp):
    """The gradient by the formulas of the header."""
    out = np.zeros_like(logits)
    for t, row in enumerate(logits):
        js = [j for j in range(hp.topk) if 0 <= idx[t, j] < row.size]
        if not js:
            continue
        s, g = scores(row, hp.score), hp.scale * dweights[t, js]
        at = idx[t, js]
        if hp.renormalise:
            w = weights_of(row, at, hp) / hp.scale if hp.scale else np.zeros(len(js))
            d = w * (g - (g * w).sum())
            if hp.score == osa.OPTIM_ROUTE_SIGMOID:
                d = d * (1 - s[at])
        elif hp.score == osa.OPTIM_ROUTE_SIGMOID:
            d = g * s[at] * (1 - s[at])
        else:
            out[t] -= s * (g * s[at]).sum()
            d = g * s[at]
        for e, x in zip(at, d):
            out[t, e] += x
    return out


def rows_of(idx, experts):
    """(offsets, place, order): the choices by expert, each expert's in order."""
    flat = idx.reshape(-1)
    by = [[i for i, e in enumerate(flat) if e == x] for x in range(experts)]
    order = np.full(flat.size, -1, np.int32)
    all_ = [i for run in by for i in run]
    order[:len(all_)] = all_
    place = np.full(flat.size, -1, np.int32)
    place[all_] = np.arange(len(all_))
    return np.cumsum([0] + [len(r) for r in by]).astype(np.int32), place.reshape(idx.shape), order


def philox(block, step, site, seed):
    """Philox4x32-10 in Python's whole numbers."""
    m = 0xFFFFFFFF
    a, b, c, d, k0, k1 = block & m, block >> 32, step & m, site, seed & m, seed >> 32
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (y >> 32) ^ b ^ k0, y & m, (x >> 32) ^ d ^ k1, x & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return a, b, c, d


def kept(n, p, seed, step, site, first):
    """The factor of each of n elements: 0, or one over the share kept."""
    bar = min(65535, math.floor(65536 * p + 0.5))
    out, words, at = np.zeros(n), None, -1
    for i in range(n):
        q = first + i
        if q >> 3 != at:
            at = q >> 3
            words = philox(at, step, site, seed)
        r = words[(q & 7) >> 1] >> (16 * (q & 1)) & 0xFFFF
        out[i] = 0.0 if r < bar else 65536 / (65536 - bar)
    return out


def apart(rows, cols, dtype, by, gen=None, fill=float("nan")):
    """A [rows, cols] view of a matrix whose rows lie `by` elements further apart
    and begin one element in; what lies between is `fill`."""
    whole = torch.full((rows * (cols + by) + 1,), fill, dtype=dtype, device=DEV)
    view = whole[1:].view(rows, cols + by)[:, :cols]
    return whole, view


def spread(matrix, by):
    """The same values in a matrix whose rows lie apart (see `apart`)."""
    whole, view = apart(matrix.size(0), matrix.size(1), matrix.dtype, by)
    view.copy_(matrix)
    return view
