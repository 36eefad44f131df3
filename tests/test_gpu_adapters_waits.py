"""Bounded waits of the launches that compute V for many rows and that write D beside a
product: the producer stops early, every wait runs out and is recorded, the next call is right.
And inputs that change from call to call while the launches of those forms overlap."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev
from test_gpu_adapters import BF, Problem

pytestmark = pytest.mark.gpu


def stalls(call, p, after):
    """call(D, ws) with producers that stop after so many loads, then as usual."""
    T, N = p.sizes[:2]
    want, ws = torch.empty(T, N, dtype=BF, device=dev()), p.workspace()
    call(want, ws)
    assert dg.dgemm_query_device_status(ws) == 0
    D = torch.empty_like(want)
    with dg.overrides(wait_limit_ns=2_000_000, stall_after_loads=after):
        call(D, ws)
        torch.cuda.synchronize()
    assert dg.dgemm_query_device_status(ws) != 0
    call(D, ws)
    assert dg.dgemm_query_device_status(ws) == 0 and torch.equal(D, want)


@pytest.mark.parametrize("after", [0, 1])
@pytest.mark.parametrize("K,order", [(136, "runs"), (1024, "runs"), (2056, "mixed")])       # 1, 4 and 8 CTAs share K
@pytest.mark.parametrize("form", [0, 1])
def test_v_of_many_rows(K, order, after, form):
    p = Problem(1100, 264, K, 16, 6, order=order)
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    with dg.overrides(cta_pair=form):
        stalls(lambda D, ws: dg.dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, ws=ws), p, after)


@pytest.mark.parametrize("T,r,order", [(300, 16, "mixed"), (300, 24, "one"), (300, 32, "one"), (1100, 128, "runs")])
@pytest.mark.parametrize("after", [0, 1, 2])
@pytest.mark.parametrize("beside", [True, False])
def test_beside_a_product(T, r, order, after, beside):
    # (one adapter of rank 24 or 32 is one load of B a tile beside one of C)
    p = Problem(T, 520, 64, r, 4, order=order)
    X, A, B, ids, scale = p.on_gpu("X", "A", "B", "ids", "scale")
    C = p.C.to(BF).to(dev()) if beside else None
    if order == "one" and after >= 1 + beside:
        return                                  # there are no more loads to stop before
    with dg.overrides(cta_pair=1):
        stalls(lambda D, ws: dg.dgemm_adapter_add(X, A, B, ids, D, C=C, scale=scale, act="silu", ws=ws), p, after)


@pytest.mark.parametrize("T", [700, 1100])
@pytest.mark.parametrize("product", [True, False])
def test_inputs_written_just_before_and_after_the_call(T, product):
    p = Problem(T, 1032, 2048, 16, 4, order="runs")
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    ws, C2 = p.workspace(), torch.empty(T, 1032, dtype=BF, device=dev())
    make = lambda i, *s: torch.randn(*s, generator=torch.Generator().manual_seed(i)).to(BF).to(dev())
    given = [(make(i, T, 2048), make(i + 50, T, 1032), make(i + 100, 4, 1032, 16)) for i in range(6)]

    def call(x, c, b):
        D = torch.empty(T, 1032, dtype=BF, device=dev())
        if product:
            return dg.dgemm_adapter_bf16(x, W, A, b, ids, D, scale=scale, ws=ws)
        return dg.dgemm_adapter_add(x, A, b, ids, D, C=c, scale=scale, ws=ws)

    want = []
    for g in given:
        want.append(call(*g))
        torch.cuda.synchronize()
    X2, B2, got = torch.empty_like(X), torch.empty_like(B), []
    for x, c, b in given:
        X2.copy_(x)
        C2.copy_(c)
        B2.copy_(b)
        got.append(call(X2, C2, B2))
    torch.cuda.synchronize()
    assert dg.dgemm_query_device_status(ws) == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
