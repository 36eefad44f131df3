"""The example block (examples/moe_block.py) against float64, stage by stage: each
stage's reference takes the stage's own inputs, so that every bound is one operator's."""
import os
import sys

import pytest
import torch

import dense_gemm_persistent_gb300 as dg
import experts_ref as ref
from gpu_util import dev, status_ok

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from moe_block import MoEBlock  # noqa: E402

pytestmark = pytest.mark.gpu


def close(got, want, tol):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [1, 5, 130])
def test_block(T, int8):
    b = MoEBlock(256, 192, 12, 3, 160, int8=int8, device=dev(), seed=T)
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, 256, generator=g).to(torch.bfloat16)
    out = torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device=dev())
    b(X.to(dev()), out)
    assert status_ok(b.ws)
    R = T * 3
    ids, w, offsets, row_token, slot_row = ref.route(b.logits[:T].cpu(), 3, True)
    assert b.ids[:T].tolist() == ids and b.offsets.tolist() == offsets
    assert b.row_token[:R].tolist() == row_token and b.slot_row[:T].tolist() == slot_row
    q, s = ref.quantize(X)
    assert torch.equal(b.codes[:T].cpu(), q) and torch.equal(b.scales[:T].cpu(), s)
    cpu = lambda t: t.cpu()
    rows = torch.tensor(row_token)
    if int8:
        want, tol = ref.grouped(q, cpu(b.up), offsets, a_rows=rows, a_scale=s, b_scale=cpu(b.up_scale), act="swiglu")
        close(b.inner[:R], want, tol)
        q2, s2 = ref.quantize(cpu(b.inner[:R]))
        assert torch.equal(b.inner_codes[:R].cpu(), q2) and torch.equal(b.inner_scales[:R].cpu(), s2)
        want, tol = ref.grouped(q2, cpu(b.down), offsets, a_scale=s2, b_scale=cpu(b.down_scale))
    else:
        want, tol = ref.grouped(X, cpu(b.up), offsets, a_rows=rows, act="swiglu")
        close(b.inner[:R], want, tol)
        want, tol = ref.grouped(cpu(b.inner[:R]), cpu(b.down), offsets)
    close(b.rows[:R], want, tol)
    want, tol = ref.grouped(q, cpu(b.shared)[None], [0, T], a_scale=s, b_scale=cpu(b.shared_scale)[None])
    close(b.from_shared[:T], want, tol)
    want, tol = ref.combine(cpu(b.rows[:R]), torch.tensor(slot_row), cpu(b.weights[:T]), cpu(b.from_shared[:T]))
    close(out, want, tol + (want.abs() + tol) * 2.0 ** -8 + 1e-37)


def test_block_in_a_cuda_graph():
    """The calls neither synchronise nor allocate: the block replays from a CUDA graph with
    another routing in the same buffers."""
    b = MoEBlock(256, 128, 8, 2, 64, device=dev())
    X = torch.randn(64, 256, device=dev()).to(torch.bfloat16)
    out = torch.empty_like(X)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b(X, out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b(X, out)
    X.copy_(torch.randn(64, 256, device=dev()))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    b(X, out)
    torch.cuda.synchronize()
    assert status_ok(b.ws) and torch.equal(got, out)
