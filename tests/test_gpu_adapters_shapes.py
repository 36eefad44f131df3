"""The low-rank adapters where a call has no depth, or a result has other rows than B's
channels: results and what lies around them."""
import pytest
import torch

import adapters_ref as ref
import dense_gemm_persistent_gb300 as dg
from gpu_util import dev
from test_gpu_adapters import BF, F32, Problem, close, form  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N", [(5, 256), (300, 256), (300, 260), (700, 528), (4096, 8192)])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_no_depth_and_rows_around(form, T, N, out, act):  # noqa: F811
    p = Problem(T, N, 0, 8, 3, with_bias=True)
    wide = N // 2 if act == "swiglu" else N
    room = torch.full((2 * T + 16, wide), 7.0, dtype=out, device=dev())     # (rows of N channels would still end inside)
    got = p.project(act, out, D=room[8:T + 8])
    row = Problem(1, N, 0, 8, 3)
    row.bias = p.bias
    want = ref.adapters(row.X, row.A, row.B, row.ids, W=row.W, bias=row.bias, act=act, out_dtype=out)
    assert torch.equal(got.cpu(), got[:1].cpu().expand(T, wide))            # (every row is the bias through the activation)
    close(got[:1], want)
    assert bool((room[:8] == 7).all()) and bool((room[T + 8:] == 7).all())


@pytest.mark.parametrize("T", [5, 300, 700])
def test_no_adapters_in_bf16(form, T):  # noqa: F811
    p = Problem(T, 264, 136, 8, 0, with_bias=True)
    for c in (BF, None):
        C = None if c is None else p.C.to(BF)
        close(p.add("silu", BF, c), ref.adapters(p.X, p.A, p.B, p.ids, C=C, bias=p.bias, act="silu"))
