"""NaN and infinities through the activations of the expert and int8 products: NaN stays
NaN under every one of them, and the entries beside it stay clean."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def operands(kind, R, N, K):
    """One expert whose products are 0, so that D = act(bias)."""
    t = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[kind]
    A, B = torch.ones(R, K).to(t).to(dev()), torch.zeros(1, N, K).to(t).to(dev())
    return A, B, torch.ones(R, device=dev()), torch.ones(1, N, device=dev()), torch.tensor([0, R], dtype=torch.int32, device=dev())


def product(kind, R, N, K, bias, act, D):
    A, B, sa, sb, offsets = operands(kind, R, N, K)
    if kind == "bf16":
        dg.dgemm_grouped_bf16(A, B, offsets, D, bias=bias, act=act)
    elif kind == "fp8":
        dg.dgemm_grouped_fp8_scaled(A, B, sa, sb, offsets, D, bias=bias, act=act)
    else:
        dg.dgemm_grouped_int8_scaled(A, B, sa, sb, offsets, D, bias=bias, act=act)
    assert status_ok()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("R", [1, 2, 40, 200])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_nan_stays_nan(kind, R, act, out):
    N = 130
    bias = torch.linspace(-2, 2, N)[None].contiguous()
    bias[0, ::7] = NAN
    D = torch.zeros(R, N, dtype=out, device=dev())
    product(kind, R, N, 64, bias.to(dev()), act, D)
    assert torch.equal(torch.isnan(D.cpu()), torch.isnan(bias).expand(R, -1))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("R", [1, 2, 40, 200])
def test_nan_stays_nan_gated(kind, R):
    """A NaN of either half spoils its own channel only."""
    half = 70
    bias = torch.linspace(-2, 2, 2 * half)[None].contiguous()
    bias[0, 5], bias[0, half + 9] = NAN, NAN
    D = torch.zeros(R, half, device=dev())
    product(kind, R, 2 * half, 64, bias.to(dev()), "swiglu", D)
    want = torch.zeros(R, half, dtype=torch.bool)
    want[:, 5] = want[:, 9] = True
    assert torch.equal(torch.isnan(D.cpu()), want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("R", [1, 2, 40, 200])
def test_relu_of_infinities_and_zeros(kind, R):
    bias = torch.tensor([[INF, -INF, 0.0, -0.0, 3.5, -3.5, 1e-40, -1e-40]])
    D = torch.full((R, 8), 7.0, device=dev())
    product(kind, R, 8, 64, bias.to(dev()), "relu", D)
    assert torch.equal(D.cpu(), torch.tensor([[INF, 0, 0, 0, 3.5, 0, 1e-40, 0]]).expand(R, -1))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("M", [1, 2, 40, 200])
def test_nan_row_scale_of_the_int8_layer(M, act):
    """A row whose scale is NaN is NaN throughout; the other rows are what they are without it."""
    g = torch.Generator().manual_seed(M)
    A, B = torch.randint(-127, 128, (M, 128), generator=g).to(torch.int8).to(dev()), torch.randint(-127, 128, (96, 128), generator=g).to(torch.int8).to(dev())
    sa, sb = torch.full((M,), 1e-3, device=dev()), torch.full((96,), 1e-2, device=dev())
    clean, D = torch.empty(M, 96, device=dev()), torch.empty(M, 96, device=dev())
    dg.dgemm_int8_scaled(A, B, sa, sb, clean, act=act)
    sa[M - 1] = NAN
    dg.dgemm_int8_scaled(A, B, sa, sb, D, act=act)
    assert status_ok()
    assert torch.equal(D[:M - 1], clean[:M - 1]) and bool(torch.isnan(D[M - 1]).all())
