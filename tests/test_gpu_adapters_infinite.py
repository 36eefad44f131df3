"""Infinities of V and of B in the same term of the low-rank adapters: an infinity times an
infinity is one, in every form, and stays with its request's rows."""
import pytest
import torch

import adapters_ref as ref
from test_gpu_adapters import BF, F32, Problem, form  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def calls(p):
    return [(lambda: p.project(out=F32), dict(W=p.W), F32), (lambda: p.project(), dict(W=p.W), BF),
            (lambda: p.add(out=BF, c=BF), dict(C=p.C.to(BF)), BF), (lambda: p.add(out=F32, c=F32), dict(C=p.C), F32)]


def same(got, want, out):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)].to(out))
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))


@pytest.mark.parametrize("T,N,K,r,order", [(8, 264, 256, 16, "mixed"), (60, 130, 64, 32, "mixed"), (200, 264, 64, 24, "runs"),
                                           (300, 264, 72, 32, "one"), (520, 264, 256, 16, "mixed"), (400, 136, 64, 128, "one"),
                                           (1100, 136, 136, 16, "runs")])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_both_factors(form, T, N, K, r, order, bad):  # noqa: F811
    p = Problem(T, N, K, r, 6, order=order)
    a = 5 if order == "one" else 2
    hit = p.ids == a
    assert bool(hit.any())
    p.A[a, 3, 5] = INF                              # V[t, 3] is +-inf by the sign of X[t, 5], in all rows of the request
    p.X[:, 5] = torch.where(p.X[:, 5] == 0, torch.ones_like(p.X[:, 5]), p.X[:, 5])
    p.B[a, :, 3] = p.B[a, :, 3].abs() + 0.5
    clean = [call() for call, _, _ in calls(p)]
    p.B[a, 7, 3] = p.B[a, N - 1, 3] = bad           # the same term's other factor
    p.B[a, 100, 0] = bad                            # and beside it
    for (call, beside, out), was in zip(calls(p), clean):
        got = call().cpu()
        same(got[hit], ref.adapters(p.X, p.A, p.B, p.ids, **beside, scale=p.scale, out_dtype=out)[0][hit], out)
        assert torch.equal(got[~hit], was.cpu()[~hit])


@pytest.mark.parametrize("T,r", [(8, 16), (300, 32), (520, 24)])
@pytest.mark.parametrize("x", [INF, -INF])
def test_an_infinite_row_meets_an_infinite_adapter(form, T, r, x):  # noqa: F811
    p = Problem(T, 264, 256, r, 6, order="mixed")
    p.ids[4] = 2
    p.A[2, :, 0] = 1.0
    p.B[2] = p.B[2].abs() + 0.5
    p.W[:, 0] = 1.0
    clean = [call() for call, _, _ in calls(p)]
    p.X[4, 0] = x
    p.B[2, 9, 1] = INF
    p.B[2, 77, 2] = -INF
    hit = p.ids == 2
    for (call, beside, out), was in zip(calls(p), clean):
        got = call().cpu()
        want = ref.adapters(p.X, p.A, p.B, p.ids, **beside, scale=p.scale, out_dtype=out)[0]
        assert bool((want[4, :9] == x).all()) and want[4, 9] == x and bool(want[4, 77].isnan())
        same(got[hit], want[hit], out)
        assert torch.equal(got[~hit], was.cpu()[~hit])
