"""The routed-expert and 8-bit integer operators beyond 2^31 elements of each operand: rows by
index, weights, outputs, combined and quantised rows. Small integers keep every sum exact, so
sampled rows around and past the limit are compared bit for bit."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

TWO31 = 2 ** 31
BF, I8, E4M3 = torch.bfloat16, torch.int8, torch.float8_e4m3fn
TYPES = {"bf16": BF, "fp8": E4M3, "int8": I8}


@pytest.fixture(autouse=True)
def memory():
    """Hands the multi-gigabyte buffers back before the next test."""
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def small_ints(seed, *shape, dtype):
    """Integers -3..3 on the device (each is exact in every type)."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randint(-3, 4, shape, generator=g, device=dev(), dtype=I8)
    return x if dtype == I8 else x.to(dtype)


def f64(x):
    return x.cpu().to(torch.float64)


def grouped(kind, A, B, offsets, D, **kw):
    offsets = torch.tensor(offsets, dtype=torch.int32, device=dev())
    if kind == "bf16":
        dg.dgemm_grouped_bf16(A, B, offsets, D, **kw)
    else:
        f = dg.dgemm_grouped_fp8_scaled if kind == "fp8" else dg.dgemm_grouped_int8_scaled
        one = lambda *s: torch.ones(*s, device=dev())
        f(A, B, one(A.shape[0]), one(*B.shape[:2]), offsets, D, **kw)
    assert status_ok()


@pytest.mark.parametrize("kind,pair", [("bf16", 1), ("bf16", 0), ("fp8", 1), ("int8", 1), ("int8", 0)])
def test_output_rows(kind, pair):
    R, N, K = 66048, 32776, 16
    assert (R - 512) * N > TWO31
    A, B = small_ints(1, R, K, dtype=TYPES[kind]), small_ints(2, 2, N, K, dtype=TYPES[kind])
    D = torch.full((R, N), 99.0, dtype=BF, device=dev())
    with dg.overrides(cta_pair=pair):
        grouped(kind, A, B, [0, 40000, R], D)
    rows = torch.tensor([0, 39999, 40000, TWO31 // N - 1, TWO31 // N, TWO31 // N + 1, R - 300, R - 2, R - 1])
    for r in rows.tolist():
        want = f64(A[r]) @ f64(B[int(r >= 40000)]).t()
        assert torch.equal(f64(D[r]), want), r


@pytest.mark.parametrize("kind,R", [("bf16", 40), ("bf16", 200), ("fp8", 200), ("int8", 40), ("int8", 200), ("int8", 2)])
def test_rows_by_index(kind, R):
    K, N = 4096, 72
    count = TWO31 // K + 700
    A, B = small_ints(3, count, K, dtype=TYPES[kind]), small_ints(4, 1, N, K, dtype=TYPES[kind])
    g = torch.Generator().manual_seed(R)
    rows = torch.randint(count - 1400, count, (R,), generator=g)      # on both sides of the limit
    rows[0], rows[-1] = 0, count - 1
    D = torch.full((R, N), 99.0, device=dev())
    grouped(kind, A, B, [0, R], D, a_rows=rows.to(torch.int32).to(dev()))
    pick = torch.stack([A[r].to(torch.float32) for r in rows.tolist()])
    assert torch.equal(f64(D), f64(pick) @ f64(B[0]).t())


@pytest.mark.parametrize("kind,layout", [("bf16", "nk"), ("bf16", "kn"), ("fp8", "nk"), ("int8", "nk")])
@pytest.mark.parametrize("R", [16, 800])
def test_weights(kind, layout, R):
    E, N, K = 40, 8192, 6784
    assert (E - 1) * N * K > TWO31
    B = small_ints(5, E, *((N, K) if layout == "nk" else (K, N)), dtype=TYPES[kind])
    A = small_ints(6, R, K, dtype=TYPES[kind])
    last = [0] * E + [R]                                    # the last expert has every row
    half = [0] + [R // 2] * (E - 1) + [R]                   # the first and the last one
    for offsets in (last, half):
        D = torch.full((R, N), 99.0, device=dev())
        grouped(kind, A, B, offsets, D, **(dict(b_layout=layout) if kind == "bf16" else {}))
        for r in (0, R // 2 - 1, R // 2, R - 1):
            e = 0 if r < offsets[1] else E - 1
            b = f64(B[e]) if layout == "kn" else f64(B[e]).t()
            assert torch.equal(f64(D[r]), f64(A[r]) @ b), r


@pytest.mark.parametrize("M", [1, 2])
def test_one_or_two_int8_rows_of_many_channels(M):
    K = 4096
    N = TWO31 // K + 513
    A, B = small_ints(7, M, K, dtype=I8), small_ints(8, N, K, dtype=I8)
    D = torch.full((M, N), 99.0, device=dev())
    one = lambda n: torch.ones(n, device=dev())
    dg.dgemm_int8_scaled(A, B, one(M), one(N), D)
    assert status_ok()
    for at in (slice(0, 64), slice(N - 1100, N)):
        assert torch.equal(f64(D[:, at]), f64(A) @ f64(B[at]).t())


@pytest.mark.parametrize("H", [8192, 8195])
def test_combine(H):
    T = TWO31 // H + 300                                    # Y, add and out are all beyond the limit
    Y, add = small_ints(9, T, H, dtype=BF), small_ints(10, T, H, dtype=BF)
    g = torch.Generator().manual_seed(H)
    slot = torch.randperm(T, generator=g).to(torch.int32).reshape(T, 1)
    w = torch.randint(-4, 5, (T, 1), generator=g).float()
    out = torch.full((T, H), 99.0, dtype=BF, device=dev())
    dg.dgemm_combine(Y, slot.to(dev()), w.to(dev()), out, add=add)
    far = (slot[:, 0] >= TWO31 // H).nonzero()[:3, 0].tolist()
    for t in [0, TWO31 // H - 1, TWO31 // H, T - 1] + far:
        assert torch.equal(f64(out[t]), float(w[t]) * f64(Y[int(slot[t])]) + f64(add[t])), t


@pytest.mark.parametrize("K,dtype", [(8192, BF), (4096, torch.float32), (8200, BF), (1001, BF)])
def test_int8_quantize(K, dtype):
    M = TWO31 // K + 300
    X = torch.empty(M, K, dtype=dtype, device=dev())
    g = torch.Generator(device=dev()).manual_seed(K)
    step = 65536
    for m in range(0, M, step):
        X[m:m + step] = torch.randn(min(step, M - m), K, generator=g, device=dev()).to(dtype)
    q = torch.full((M, K), 99, dtype=I8, device=dev())
    s = torch.full((M,), -1.0, device=dev())
    dg.dgemm_int8_quantize(X, q, s)
    inv127 = torch.tensor(1.0) / torch.tensor(127.0)
    for m in (0, 1, TWO31 // K - 1, TWO31 // K, TWO31 // K + 1, M - 1):
        x = X[m].cpu().float()
        scale = x.abs().max() * inv127
        assert float(s[m]) == float(scale) and torch.equal(q[m].cpu(), torch.round(x / scale).to(I8)), m


def test_route_logits():
    """2.1 million tokens of 1024 logits each: the last 2048 tokens' logits lie past the limit."""
    E, k = 1024, 1
    T = TWO31 // E + 2048
    i32 = dict(dtype=torch.int32, device=dev())
    logits = torch.zeros(T, E, dtype=BF, device=dev())
    pick = torch.randint(0, E, (T,), generator=torch.Generator(device=dev()).manual_seed(11), device=dev())
    logits.scatter_(1, pick[:, None], 1.0)
    ids, slot_row = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
    weights, offsets, row_token = torch.empty(T, k, device=dev()), torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    ws = torch.empty(dg.dgemm_route_workspace_size(T, E, k), dtype=torch.uint8, device=dev())
    dg.dgemm_route(logits, k, ids, weights, offsets, row_token, slot_row, ws=ws)
    assert torch.equal(ids[:, 0].long(), pick)
    order = torch.sort(pick, stable=True).indices
    assert torch.equal(row_token.long(), order)
    assert torch.equal(slot_row[:, 0].long()[order], torch.arange(T, device=dev()))
    assert torch.equal(offsets[1:].long(), torch.bincount(pick, minlength=E).cumsum(0)) and int(offsets[0]) == 0
