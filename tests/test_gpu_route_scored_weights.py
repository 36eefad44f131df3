"""The weights of the routing by scores: far below zero, and within bounds that count the
roundings they take."""
import math

import pytest
import torch

import adapters_ref as ref
import dense_gemm_persistent_gb300 as dg
from gpu_util import dev
from test_gpu_route_scored import BF, F32, gen, outputs

pytestmark = pytest.mark.gpu


def weights_of(x, k, **how):
    T, E = x.shape
    out = outputs(T, E, k)
    ws = torch.empty(max(256, dg.dgemm_route_workspace_size(T, E, k)), dtype=torch.uint8, device=dev())
    dg.dgemm_route_scored(x.to(dev()), k, *out, ws=ws, **how)
    return out[0].cpu(), out[1].cpu().double()


@pytest.mark.parametrize("k", [1, 4, 8, 32])
@pytest.mark.parametrize("bias", [False, True])
def test_sigmoid_scores_below_the_normal_numbers(k, bias):
    # s = e^x to 2^-24 here. All of a row's scores are the same, or fall from one to the next; while their sum is 2^-126
    # or more a weight is its part of the sum, and below that s 2^126
    starts = [-80.0, -87.0, -87.5, -88.0, -88.6, -89.0, -90.0, -91.0, -95.0, -103.0, -110.0, -3.0e38]
    rows = [[s - step * e for e in range(48)] for s in starts for step in (0.0, 0.03, 0.7)]
    x = torch.tensor(rows)
    ids, got = weights_of(x, k, score="sigmoid", bias=torch.zeros(48, device=dev()) if bias else None, scale=2.0)
    for t, row in enumerate(x.double().tolist()):
        # (a bias of zero leaves scores that are equal in FP64, 0, in the experts' order)
        assert ids[t].tolist() == list(range(k))
        s = [math.exp(v) if v > -700 else 0.0 for v in row[:k]]
        total = max(sum(s), 2.0 ** -126)
        want = torch.tensor([2.0 * v / total for v in s], dtype=torch.float64)
        # exponentials of differences up to 33 and of 130 (halved, then squared), 5 sums, quotient, product: under 2^-16
        assert bool(((got[t] - want).abs() <= want * 2.0 ** -16 + 1e-30).all()), (t, got[t], want)


@pytest.mark.parametrize("T,E,k", [(200, 64, 6), (90, 256, 8), (40, 1024, 32)])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("bias", [False, True])
def test_weights_to_the_roundings_they_take(T, E, k, score, renorm, bias):
    """In units of 2^-24: an exponential 4 (2 in the last place) and the rounding of its argument |d|, |d| the distance
    from the row's largest logit, or of sigmoid from 0; a quotient 4 (__fdividef), a sum with 1 and a product 1 each; a sum
    over k lanes 5 more. The softmax's own sum: special-function exponentials 4, their arguments' roundings weighted by the
    terms up to 1.5 ln 1024 = 11, E / 32 and 5 additions, and its full quotient 1."""
    g = gen(T + E)
    x = 3.0 * torch.randn(T, E, generator=g)
    b = (0.1 * torch.randn(E, generator=g)).to(dev()) if bias else None
    ids, got = weights_of(x, k, score=score, bias=b, renormalize=renorm, scale=2.5)
    v = x.double()
    p = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
    s = torch.gather(p, 1, ids.long())
    d = torch.gather(v.amax(1, keepdim=True) - v if score == "softmax" else v.abs(), 1, ids.long())
    if renorm:
        want = 2.5 * s / s.sum(1, keepdim=True)
        units = 2 * (4 + d.amax(1, keepdim=True) + 1 + 4) + 5 + 4 + 1
    else:
        want = 2.5 * s
        units = 4 + d + (4 + 11 + max(2, E // 32) + 5 + 1 + 1 if score == "softmax" else 1 + 4) + 1
    assert bool(((got - want).abs() <= want * units * 2.0 ** -24).all()), float(((got - want).abs() / want / units).max() * 2 ** 24)
