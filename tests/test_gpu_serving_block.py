"""The example block with experts chosen by scores and the adapters of many requests on its shared
layer, stage by stage against float64, and replayed from a CUDA graph."""
import os
import sys

import pytest
import torch

import adapters_ref
import dense_gemm_persistent_gb300 as dg
import experts_ref as ref
from gpu_util import dev, status_ok

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from moe_block import MoEBlock  # noqa: E402

pytestmark = pytest.mark.gpu


def close(got, want, tol):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def block(seed, int8=False):
    return MoEBlock(256, 192, 16, 3, 400, int8=int8, scored=True, groups=4, groups_kept=2, adapters=5, rank=16, device=dev(), seed=seed)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [1, 7, 390])
def test_block(T, int8):
    b = block(T, int8)
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, 256, generator=g).to(torch.bfloat16)
    requests = torch.randint(-1, 5, (T,), generator=g).sort().values.to(torch.int32)
    out = torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device=dev())
    b(X.to(dev()), out, requests.to(dev()))
    assert status_ok(b.ws)
    ids, w, offsets, row_token, slot_row = adapters_ref.route_scored(b.logits[:T].cpu(), 3, "sigmoid", b.balance.cpu(), 4, 2, "top2",
                                                                     True, 2.5)
    assert b.ids[:T].tolist() == ids and b.offsets.tolist() == offsets
    assert b.row_token[:T * 3].tolist() == row_token and b.slot_row[:T].tolist() == slot_row
    q, s = ref.quantize(X)
    cpu = lambda t: t.cpu()
    # the shared layer: the int8 product (its own bound), rounded to BF16, then the adapters in place
    base, base_tol = ref.grouped(q, cpu(b.shared)[None], [0, T], a_scale=s, b_scale=cpu(b.shared_scale)[None])
    want, tol = adapters_ref.adapters(X, cpu(b.low), cpu(b.high), requests, C=base, scale=cpu(b.adapter_scale))
    close(b.from_shared[:T], want, tol + base_tol * (1 + 2.0 ** -8))
    want, tol = ref.combine(cpu(b.rows[:T * 3]), torch.tensor(slot_row), cpu(b.weights[:T]), cpu(b.from_shared[:T]))
    close(out, want, tol + (want.abs() + tol) * 2.0 ** -8 + 1e-37)


def test_block_in_a_cuda_graph():
    b = block(3)
    X = torch.randn(390, 256, device=dev()).to(torch.bfloat16)
    requests = (torch.arange(390, device=dev()) // 80).to(torch.int32)
    out = torch.empty_like(X)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b(X, out, requests)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b(X, out, requests)
    X.copy_(torch.randn(390, 256, device=dev()))
    requests.copy_(requests.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    b(X, out, requests)
    torch.cuda.synchronize()
    assert status_ok(b.ws) and torch.equal(got, out)
