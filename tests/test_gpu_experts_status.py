"""A wait that ran out stays on record in the workspace until it is queried, whatever
operators are given the same workspace in between."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

TIMEOUT = 6   # DGEMM_ERR_DEVICE_TIMEOUT


def route_into(ws, T, E, k):
    i32 = dict(dtype=torch.int32, device=dev())
    ids, slot_row = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
    weights = torch.empty(T, k, device=dev())
    offsets, row_token = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(dev())
    dg.dgemm_route(logits, k, ids, weights, offsets, row_token, slot_row, ws=ws)
    want = torch.topk(logits, k, dim=1).indices
    assert torch.equal(ids.long(), want)
    assert torch.equal(offsets.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long),
                                                        torch.bincount(want.cpu().reshape(-1), minlength=E).cumsum(0)]))


@pytest.mark.parametrize("T,E,k", [(64, 64, 4), (65, 64, 4), (2000, 64, 4), (2000, 256, 8)])
def test_routing_keeps_a_recorded_timeout(T, E, k):
    ws = torch.full((max(256, dg.dgemm_route_workspace_size(T, E, k)),), 0x5A, dtype=torch.uint8, device=dev())
    A, B = torch.ones(20, 2048, dtype=torch.bfloat16, device=dev()), torch.ones(1, 300, 2048, dtype=torch.bfloat16, device=dev())
    D = torch.zeros(20, 300, device=dev())
    offsets = torch.tensor([0, 20], dtype=torch.int32, device=dev())
    with dg.overrides(stall_after_loads=2, wait_limit_ns=20_000_000):
        dg.dgemm_grouped_bf16(A, B, offsets, D, ws=ws)
    for _ in range(3):
        route_into(ws, T, E, k)
    assert dg.dgemm_query_device_status(ws) == TIMEOUT
    assert status_ok(ws)                       # the query cleared it
    dg.dgemm_grouped_bf16(A, B, offsets, D, ws=ws)
    route_into(ws, T, E, k)
    assert status_ok(ws) and bool((D == 2048).all())
