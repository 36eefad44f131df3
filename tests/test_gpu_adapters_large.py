"""The low-rank adapters beyond 2^31 elements of each operand. Small integers keep every sum exact, so sampled
rows around and past the limit are compared bit for bit."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

TWO31 = 2 ** 31
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    """Hands the multi-gigabyte buffers back before the next test."""
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def small_ints(seed, *shape, most=1):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=dev(), dtype=torch.int8).to(BF)


def want_row(t, X, A, B, ids, y):
    a = int(ids[t])
    f = lambda x: x.cpu().double()
    return y + (f(B[a]) @ (f(A[a]) @ f(X[t])) if 0 <= a < A.shape[0] else 0.0)


def run(X, A, B, ids, T, N, W=None, C=None, in_place=False):
    D = C if in_place else torch.full((T, N), 99.0, dtype=BF, device=dev())
    ws = torch.empty(dg.dgemm_adapter_workspace_size(T, N, X.shape[1], A.shape[1], A.shape[0]), dtype=torch.uint8, device=dev())
    if W is not None:
        dg.dgemm_adapter_bf16(X, W, A, B, ids, D, ws=ws)
    else:
        dg.dgemm_adapter_add(X, A, B, ids, D, C=C, ws=ws)
    assert status_ok(ws)
    return D


@pytest.mark.parametrize("N", [32776, 32777])
@pytest.mark.parametrize("product", [True, False])
def test_output_rows(N, product):
    T, K, r, L = 66048, 16, 8, 3
    assert (T - 512) * N > TWO31
    X, A, B = small_ints(1, T, K), small_ints(2, L, r, K), small_ints(3, L, N, r)
    ids = torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    W = small_ints(5, N, K) if product else None
    C = None if product else small_ints(6, T, N, most=3)
    rows = [0, 40000, TWO31 // N - 1, TWO31 // N, TWO31 // N + 1, T - 300, T - 2, T - 1]
    y = [(X[t].cpu().double() @ W.cpu().double().t()) if product else C[t].cpu().double() for t in rows]
    D = run(X, A, B, ids.to(dev()), T, N, W=W, C=C, in_place=not product)
    for t, base in zip(rows, y):
        assert torch.equal(D[t].cpu().double(), want_row(t, X, A, B, ids, base).to(BF).double()), t


@pytest.mark.parametrize("T", [6, 700])
def test_adapters_past_the_limit(T):
    L, N, K, r = 70, 262152, 131080, 128                     # A and B have more than 2^31 elements from adapter 64 on
    assert (L - 2) * N * r > TWO31
    X = small_ints(1, T, K)
    X[:, 64:] = 0
    A = torch.zeros(L, r, K, dtype=BF, device=dev())
    A[:, :, :64] = small_ints(2, L, r, 64)
    B = small_ints(3, L, N, r)
    ids = torch.tensor([L - 1, 0, L - 2, 63, 64, -1] * (T // 6 + 1), dtype=torch.int32)[:T]
    C = small_ints(4, T, N)
    D = run(X, A, B, ids.to(dev()), T, N, C=C)
    for t in range(0, T, max(1, T // 13)):
        assert torch.equal(D[t].cpu().double(), want_row(t, X[:, :64], A[:, :, :64], B, ids, C[t].cpu().double()).to(BF).double()), t


@pytest.mark.parametrize("r,N", [(8, 8), (16, 40)])
def test_many_rows(r, N):
    """Most rows of one adapter, single rows of others between them, everywhere."""
    T, K, L = 300001, 24, 40
    X, A, B = small_ints(1, T, K), small_ints(2, L, r, K), small_ints(3, L, N, r)
    g = torch.Generator().manual_seed(4)
    ids = torch.where(torch.rand(T, generator=g) < 0.02, torch.randint(-1, L, (T,), generator=g), 7).to(torch.int32)
    C = small_ints(6, T, N)
    D = run(X, A, B, ids.to(dev()), T, N, C=C)
    f = lambda x: x.cpu().double()
    Af, Bf, Xf, Cf, own = f(A), f(B), f(X), f(C), ids.long()
    V = torch.stack([(Xf[t] @ Af[own[t]].t()) if own[t] >= 0 else torch.zeros(r, dtype=torch.float64)
                     for t in (own != 7).nonzero()[:, 0].tolist()])
    want = Cf + (Xf @ Af[7].t()) @ Bf[7].t()
    for i, t in enumerate((own != 7).nonzero()[:, 0].tolist()):
        want[t] = Cf[t] + Bf[own[t]] @ V[i]
    assert torch.equal(f(D), want.to(BF).double())


def test_a_long_row():
    T, N, K, r, L = 700, 64, 3200000, 8, 2                  # X has more than 2^31 elements
    assert (T - 20) * K > TWO31
    X = torch.zeros(T, K, dtype=BF, device=dev())
    X[:, -64:] = small_ints(1, T, 64)
    A = torch.zeros(L, r, K, dtype=BF, device=dev())
    A[:, :, -64:] = small_ints(2, L, r, 64)
    B = small_ints(3, L, N, r)
    ids = torch.tensor([0, 1] * (T // 2), dtype=torch.int32)
    for form in (0, 1):
        with dg.overrides(cta_pair=form):
            D = run(X, A, B, ids.to(dev()), T, N, C=torch.zeros(T, N, dtype=BF, device=dev()))
        for t in (0, T // 2, T - 2, T - 1):
            assert torch.equal(D[t].cpu().double(), want_row(t, X[:, -64:], A[:, :, -64:], B, ids, 0.0).to(BF).double()), (form, t)
