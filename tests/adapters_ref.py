"""Float64 references of the scored routing and the low-rank adapters, written from
their definitions, and the error bounds that the kernels are held to.

Bounds of the adapters. A product of K terms on the tensor core is off by at most
(K / 8 + 4) * 2^-23 times the sum of its terms' magnitudes (experts_ref.py); in FP32
units, summed by 128 threads with two sums each and a tree, by (K / 256 + 12) * 2^-24,
which is less. V = s X A^T takes one more rounding for the scale and, on its way through
the tensor core, two BF16 numbers: the first leaves at most 2^-9 of it, the second 2^-9
of that, 2^-18 of V. The error of V goes through B by the magnitudes of B; V . B^T adds
its own 2 r terms. Two additions (adapter, bias) round once each.
"""
from __future__ import annotations

import math

import torch

import experts_ref

F64 = torch.float64


def adapters(X, A, B, ids, *, W=None, C=None, scale=None, bias=None, act="none", out_dtype=torch.bfloat16):
    """(values, bounds on the error) in float64."""
    T, K = X.shape
    L, r, _ = A.shape
    N = B.shape[1]
    x = X.to(F64)
    y = torch.zeros(T, N, dtype=F64)
    dy = torch.zeros(T, N, dtype=F64)
    if W is not None:
        y = x @ W.to(F64).t()
        dy = (x.abs() @ W.to(F64).abs().t()) * ((K / 8 + 4) * 2.0 ** -23)
    if C is not None:
        y = C.to(F64).clone()
    for t in range(T):
        a = int(ids[t])
        if not 0 <= a < L:
            continue
        s = 1.0 if scale is None else float(scale[a])
        v = s * (A[a].to(F64) @ x[t])
        dv = abs(s) * (A[a].to(F64).abs() @ x[t].abs()) * ((K / 8 + 8) * 2.0 ** -23) + v.abs() * (2.0 ** -24 + 2.0 ** -18)
        b = B[a].to(F64)
        y[t] += b @ v
        dy[t] += b.abs() @ dv + (b.abs() @ (v.abs() + dv)) * ((2 * r / 8 + 4) * 2.0 ** -23)
    dy = dy + (y.abs() + dy) * 2.0 ** -23
    if bias is not None:
        y = y + bias.to(F64)
        dy = dy + (y.abs() + bias.to(F64).abs()) * 2.0 ** -23
    if act == "swiglu":
        wide = N // 2
        g, u, dg, du = y[:, :wide], y[:, wide:], dy[:, :wide], dy[:, wide:]
        s = experts_ref.activation(g, "silu")
        v = s * u
        dv = 1.13 * dg * (u.abs() + du) + s.abs() * du + v.abs() * 2.0 ** -20
    else:
        v = experts_ref.activation(y, act)
        dv = 1.13 * dy + (v.abs() * 2.0 ** -20 if act != "none" else 0.0)
    return v, dv + (v.abs() + dv) * (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24) + 1e-37


def route_scored(x, k, score, bias, groups, kept, group_score, renorm, scale):
    """ids, weights (float64), offsets, row_token, slot_row as Python lists. x: FP32 values."""
    T, E = x.shape
    size = E // groups
    big = 3.4028234663852886e38

    def value(f):
        f = float(f)
        return None if f != f or f == -math.inf else min(f, big)

    b = [0.0] * E if bias is None else [value(f) for f in bias]
    ids, weights = [], []
    for t in range(T):
        v = [value(f) if b[e] is not None else None for e, f in enumerate(x[t])]
        some = [f for f in v if f is not None]
        if score == "sigmoid":
            s = [None if f is None else 1.0 / (1.0 + math.exp(-f)) if f > -700 else 0.0 for f in v]
        else:
            top = max(some, default=0.0)
            total = sum(math.exp(f - top) for f in some)
            s = [None if f is None else math.exp(f - top) / total for f in v]
        c = [None if f is None else f + b[e] for e, f in enumerate(s)]
        worth = []
        for g in range(groups):
            best = sorted((f for f in c[g * size:(g + 1) * size] if f is not None), reverse=True)
            worth.append(None if not best else best[0] if group_score == "max" else sum(best[:2]))
        order = sorted((g for g in range(groups) if worth[g] is not None), key=lambda g: (-worth[g], g))[:kept]
        live = [e for e in range(E) if c[e] is not None and e // size in order]
        if bias is None and (groups == 1 or group_score == "max"):
            live.sort(key=lambda e: (-v[e], e))
        else:
            live.sort(key=lambda e: (-c[e], e))
        live = live[:k]
        w = [s[e] for e in live]
        if renorm and score == "softmax":
            top = max((v[e] for e in live), default=0.0)
            w = [math.exp(v[e] - top) for e in live]
        if renorm:
            total = max(sum(w), 2.0 ** -126)
            w = [f / total for f in w]
        ids.append(live + [-1] * (k - len(live)))
        weights.append([f * scale for f in w] + [0.0] * (k - len(live)))
    pairs = sorted((ids[t][j], t, j) for t in range(T) for j in range(k) if ids[t][j] >= 0)
    offsets = [sum(1 for p in pairs if p[0] < e) for e in range(E + 1)]
    row_token = [p[1] for p in pairs] + [-1] * (T * k - len(pairs))
    slot_row = [[-1] * k for _ in range(T)]
    for r, (_, t, j) in enumerate(pairs):
        slot_row[t][j] = r
    return ids, weights, offsets, row_token, slot_row
