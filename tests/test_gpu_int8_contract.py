"""What the int8 products promise of their sums: exact integers below 2^24, the documented
bound beyond that, and for one or two rows of one set of weights (up to 74 KB of codes)
exact integers of any size, rounded once to FP32. The codes give odd sums, so that no
common factor hides a lost bit."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

FEW_BYTES = 74 * 1024     # codes of the token rows that the integer kernel holds


def near_the_top(g, rows, K):
    """Codes of 127, a few entries off by one: sums of about 16129 K, odd or even by chance."""
    x = torch.full((rows, K), 127, dtype=torch.int8)
    x[torch.rand(rows, K, generator=g) < 0.03] = 126
    return x


def run(A, B):
    D = torch.full((A.shape[0], B.shape[0]), float("nan"), device=dev())
    one = lambda n: torch.ones(n, device=dev())
    dg.dgemm_int8_scaled(A.to(dev()), B.to(dev()), one(A.shape[0]), one(B.shape[0]), D)
    assert status_ok()
    return D.cpu()


def sums(A, B):
    """Exact (below 2^53)."""
    return A.double() @ B.double().t()


@pytest.mark.parametrize("M,K", [(1, 1040), (2, 1040), (1, 6000), (2, 6000), (1, FEW_BYTES), (2, FEW_BYTES // 2)])
def test_one_or_two_rows_are_integers_rounded_once(M, K):
    g = torch.Generator().manual_seed(M + K)
    A, B = near_the_top(g, M, K), near_the_top(g, 37, K)
    want = sums(A, B)
    assert bool((want % 2 == 1).any()) and (K < 1041 or float(want.min()) > 2 ** 24)
    assert torch.equal(run(A, B), want.to(torch.float32))


@pytest.mark.parametrize("M,K", [(1, FEW_BYTES + 16), (2, FEW_BYTES // 2 + 16), (3, 6000), (8, 6000), (40, 6000), (200, 2048),
                                 (200, 20000)])
def test_more_rows_stay_within_the_bound(M, K):
    """Sums of K terms in FP32, one rounding toward zero for each instruction of 16 terms."""
    g = torch.Generator().manual_seed(M + K)
    A, B = near_the_top(g, M, K), near_the_top(g, 37, K)
    want = sums(A, B)
    assert float(want.min()) > 2 ** 24
    assert bool(((run(A, B).double() - want).abs() <= want * (K / 8 + 4) * 2.0 ** -23).all())


@pytest.mark.parametrize("M", [1, 2, 3, 8, 40, 200])
@pytest.mark.parametrize("K", [16, 528, 1024])
def test_sums_below_2_24_are_exact(M, K):
    g = torch.Generator().manual_seed(M * K)
    A, B = near_the_top(g, M, K), near_the_top(g, 130, K)
    want = sums(A, B)
    assert float(want.max()) < 2 ** 24 and bool((want % 2 == 1).any())
    assert torch.equal(run(A, B).double(), want)
    A = torch.randint(-128, 128, (M, K), generator=g).to(torch.int8)
    B = torch.randint(-128, 128, (130, K), generator=g).to(torch.int8)
    assert torch.equal(run(A, B).double(), sums(A, B))


@pytest.mark.parametrize("M", [1, 2, 5, 40, 200])
@pytest.mark.parametrize("N", [64, 137, 258])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pair", [-1, 0, 1])
def test_in_place_has_the_bits_of_out_of_place(M, N, dtype, pair):
    """C equal to D: every element is read before it, or a neighbour's store, overwrites it."""
    g = torch.Generator().manual_seed(M + N)
    A = torch.randint(-9, 10, (M, 80), generator=g).to(torch.int8).to(dev())
    B = torch.randint(-9, 10, (N, 80), generator=g).to(torch.int8).to(dev())
    sa, sb = torch.rand(M, generator=g).to(dev()), torch.rand(N, generator=g).to(dev())
    C = torch.randn(M, N, generator=g).to(dtype).to(dev())
    D, both = torch.empty_like(C), C.clone()
    with dg.overrides(cta_pair=pair):
        dg.dgemm_int8_scaled(A, B, sa, sb, D, C=C, beta=-1.5, act="gelu")
        dg.dgemm_int8_scaled(A, B, sa, sb, both, C=both, beta=-1.5, act="gelu")
    assert status_ok() and torch.equal(D, both)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_row_below_2_24_has_the_same_bits_among_any_number_of_rows(act, dtype):
    g = torch.Generator().manual_seed(5)
    A, B = near_the_top(g, 300, 1024), near_the_top(g, 150, 1024)
    A, B = A - torch.randint(0, 200, A.shape, generator=g).to(torch.int8), B - torch.randint(0, 200, B.shape, generator=g).to(torch.int8)
    assert float((A.abs().double() @ B.abs().double().t()).max()) < 2 ** 24
    sa, sb = 0.01 * torch.rand(300, generator=g), 0.1 * torch.rand(150, generator=g)
    C, bias = torch.randn(300, 150, generator=g).to(dtype), torch.randn(150, generator=g).to(dev())

    def rows(n):
        D = torch.empty(n, 150, dtype=dtype, device=dev())
        dg.dgemm_int8_scaled(A[:n].to(dev()), B.to(dev()), sa[:n].to(dev()), sb.to(dev()), D, C=C[:n].to(dev()), alpha=0.7, beta=0.3,
                             bias=bias, act=act)
        assert status_ok()
        return D
    whole = rows(300)
    for n in (1, 2, 3, 64, 65, 192, 193):
        assert torch.equal(rows(n), whole[:n])
