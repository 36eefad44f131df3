"""Float64 references of the routed-expert and 8-bit integer operators, written from
their definitions with plain loops over tokens and groups, and the error bounds
that their kernels are held to.

Bounds. A product of K terms summed in FP32 by the tensor core (which rounds
toward zero, one rounding per instruction of 16 or 32 terms, plus the terms'
own alignment) is off by at most (K / 8 + 4) * 2^-23 times the sum of the terms'
magnitudes; scales, bias and alpha add a few roundings of 2^-24 each. An activation
passes an error of its argument on with a slope of at most 1.13, and adds 2^-20 of
its value (fast exponential and division). One rounding to the output type
follows: 2^-8 relative for BF16 (8 significant bits), 2^-24 for FP32.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def activation(y, act):
    if act == "relu":
        return torch.clamp(y, min=0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y / math.sqrt(2.0)))
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    assert act == "none"
    return y


def grouped(A, B, bounds, *, a_rows=None, layout="nk", a_scale=None, b_scale=None, bias=None, act="none", alpha=1.0,
            out_dtype=torch.bfloat16):
    """(values [R,wide], bounds on the error) in float64; rows outside every group are
    NaN. bounds: list of E + 1 row offsets."""
    A64, B64 = A.to(F64), B.to(F64)
    E = B64.shape[0]
    N, K = (B64.shape[1], B64.shape[2]) if layout == "nk" else (B64.shape[2], B64.shape[1])
    R = A64.shape[0] if a_rows is None else len(a_rows)
    wide = N // 2 if act == "swiglu" else N
    out = torch.full((R, wide), float("nan"), dtype=F64)
    tol = torch.zeros(R, wide, dtype=F64)
    for e in range(E):
        b = B64[e].t() if layout == "nk" else B64[e]          # [K,N]
        for r in range(max(0, min(bounds[e], R)), max(0, min(bounds[e + 1], R))):
            a = r if a_rows is None else int(a_rows[r])
            inside = 0 <= a < A64.shape[0]
            row = A64[a] if inside else torch.zeros(K, dtype=F64)
            scale = torch.full((N,), float(alpha), dtype=F64)
            if a_scale is not None:
                scale = scale * (float(a_scale[a]) if inside else 0.0) * b_scale[e].to(F64)
            y = (row @ b) * scale
            size = (row.abs() @ b.abs()) * scale.abs()
            dy = size * ((K / 8 + 4) * 2.0 ** -23 + 4 * 2.0 ** -24)
            if bias is not None:
                y = y + bias[e].to(F64)
                dy = dy + (y.abs() + bias[e].to(F64).abs()) * 2.0 ** -23
            if act == "swiglu":
                g, u, dg, du = y[:wide], y[wide:], dy[:wide], dy[wide:]
                s = activation(g, "silu")
                v = s * u
                dv = 1.13 * dg * (u.abs() + du) + s.abs() * du + v.abs() * 2.0 ** -20
            else:
                v = activation(y, act)
                dv = 1.13 * dy + (v.abs() * 2.0 ** -20 if act != "none" else 0.0)
            out[r] = v
            tol[r] = dv + (v.abs() + dv) * (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24) + 1e-37
    return out, tol


def route(x, k, renorm):
    """ids, weights (float64), offsets, row_token, slot_row as Python lists."""
    T, E = x.shape
    ids, weights = [], []
    for t in range(T):
        v = []
        for e in range(E):
            f = float(x[t, e])
            if f == math.inf:
                f = 3.4028234663852886e38
            v.append(None if f != f or f == -math.inf else f)
        order = sorted((e for e in range(E) if v[e] is not None), key=lambda e: (-v[e], e))[:k]
        base = v[order[0]] if order else 0.0
        p = [math.exp(v[e] - base) for e in order]
        total = sum(p) if renorm else sum(math.exp(f - base) for f in v if f is not None)
        ids.append(order + [-1] * (k - len(order)))
        weights.append([q / total for q in p] + [0.0] * (k - len(order)))
    pairs = sorted((ids[t][j], t, j) for t in range(T) for j in range(k) if ids[t][j] >= 0)
    offsets = [sum(1 for p in pairs if p[0] < e) for e in range(E + 1)]
    row_token = [p[1] for p in pairs] + [-1] * (T * k - len(pairs))
    slot_row = [[-1] * k for _ in range(T)]
    for r, (_, t, j) in enumerate(pairs):
        slot_row[t][j] = r
    return ids, weights, offsets, row_token, slot_row


def combine(Y, slot_row, weights, add=None):
    R = Y.shape[0]
    T, k = slot_row.shape
    out = torch.zeros(T, Y.shape[1], dtype=F64) if add is None else add.to(F64).clone()
    size = out.abs()
    for t in range(T):
        for j in range(k):
            r = int(slot_row[t, j])
            if 0 <= r < R:
                term = float(weights[t, j]) * Y[r].to(F64)
                out[t] += term
                size[t] += term.abs()
    return out, size * (k + 2) * 2.0 ** -24


def quantize(X):
    """int8 codes and scales: the scale, a product with the FP32 number 1 / 127, and the
    quotient are FP32 numbers by definition."""
    x = X.to(torch.float32)
    finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    inv127 = torch.tensor(1.0) / torch.tensor(127.0)
    s = (finite.amax(1) if x.shape[1] else torch.zeros(x.shape[0])) * inv127
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = torch.round(x / s[:, None])
    q = torch.where(torch.isnan(x), torch.zeros_like(q), torch.clamp(q, -127, 127))
    return q.to(torch.int8), s
