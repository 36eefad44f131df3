"""How exact V = s X A^T is that the adapters multiply by B. Every sum of these inputs is
exact in FP32, so what is left is the form V is kept in: FP32 for few rows, two BF16
numbers for the tensor core."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def call(X, A, B, ids, W, C, form):
    T, K = X.shape
    L, r, _ = A.shape
    N = B.shape[1]
    X, A, B, ids = (t.to(dev()) for t in (X, A, B, ids))
    D = torch.full((T, N), float("nan"), device=dev())
    ws = torch.full((dg.dgemm_adapter_workspace_size(T, N, K, r, L),), 0xA5, dtype=torch.uint8, device=dev())
    with dg.overrides(cta_pair=form):
        if W is not None:
            dg.dgemm_adapter_bf16(X, W.to(dev()), A, B, ids, D, ws=ws)
        else:
            dg.dgemm_adapter_add(X, A, B, ids, D, C=None if C is None else C.to(dev()), ws=ws)
    assert status_ok(ws)
    return D.cpu().to(F64)


def check(got, want, form):
    if form == 0:
        assert torch.equal(got, want)
    else:           # V = first + second: 8 significant bits each, 2^-8 of V and 2^-9 of that
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -17).all())


@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("product", [True, False])
def test_a_number_between_two_sums_of_two(form, product):
    # V = 1 + 2^-9 + 2^-17: the first BF16 number is 1, and 2^-9 + 2^-17 lies between two others
    X, A, B = torch.zeros(3, 8, dtype=BF), torch.zeros(1, 8, 8, dtype=BF), torch.zeros(1, 16, 8, dtype=BF)
    X[:, 0], X[:, 1], X[:, 2] = 1.0, 2.0 ** -9, 2.0 ** -17
    A[0, 3] = 1.0
    B[0, :, 3] = 1.0
    zero = torch.zeros(3, 16)
    got = call(X, A, B, torch.zeros(3, dtype=torch.int32), torch.zeros(16, 8, dtype=BF) if product else None, zero, form)
    check(got, torch.full((3, 16), 1.0 + 2.0 ** -9 + 2.0 ** -17, dtype=F64), form)


@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("T,N,K,r,L", [(1, 40, 128, 8, 1), (48, 264, 136, 32, 9), (64, 130, 264, 128, 5), (300, 129, 72, 24, 4),
                                       (1100, 264, 264, 16, 6), (1100, 136, 1032, 64, 3)])
@pytest.mark.parametrize("product", [True, False])
def test_numbers_of_24_bits(form, T, N, K, r, L, product):
    # V is a sum of three 8-bit numbers, 2^0, 2^-8 and 2^-16 of the first's size; a row of B takes one of them
    g = torch.Generator().manual_seed(T + N + K + r + L)
    ints = lambda lo, hi: torch.randint(lo, hi, (L, r), generator=g).to(F32)
    sign = lambda: torch.randint(0, 2, (L, r), generator=g).to(F32) * 2 - 1
    A = torch.zeros(L, r, K)
    for k, part in enumerate((ints(129, 250), sign() * ints(128, 256), sign() * ints(128, 256))):
        A[:, :, K - 3 + k] = part * 2.0 ** (-7 - 8 * k)
    A = A.to(BF)
    size = 2.0 ** torch.randint(-3, 4, (T, 1), generator=g).to(F32)
    X = torch.zeros(T, K)
    X[:, K - 3:] = size
    X[:, :K - 3] = torch.randint(-2, 3, (T, K - 3), generator=g)              # (beside zeros of A)
    B = torch.zeros(L, N, r)
    B[:, torch.arange(N), torch.arange(N) % r] = 1.0
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
    V = A.to(F64).sum(2)
    want = torch.where((ids >= 0)[:, None], V[ids.long().clamp(min=0)][:, torch.arange(N) % r] * size.to(F64), 0.0)
    W = torch.zeros(N, K, dtype=BF) if product else None
    check(call(X.to(BF), A, B.to(BF), ids, W, None, form), want, form)
