"""The low-rank adapters against the float64 definition (tests/adapters_ref.py), at the
sizes and inputs where they can go wrong. Every tolerance is the bound derived there."""
import pytest
import torch

import adapters_ref as ref
import dense_gemm_persistent_gb300 as dg
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(params=[None, 0, 1], ids=["chosen", "few", "prompt"])
def form(request):
    """Tiles of 64 rows, the CTA pairs' tiles, or the library's choice between them."""
    if request.param is None:
        yield
    else:
        with dg.overrides(cta_pair=request.param):
            yield


class Problem:
    def __init__(self, T, N, K, r, L, seed=0, order="mixed", with_scale=True, with_bias=False):
        g = torch.Generator().manual_seed(seed * 1000003 + T * 7 + N * 5 + K * 3 + r + L)
        randn = lambda *s: torch.randn(*s, generator=g)
        self.X = (randn(T, K) * torch.exp(0.5 * randn(T, 1))).to(BF)
        self.W = (randn(N, K) * max(K, 1) ** -0.5).to(BF)
        self.A = (randn(L, r, K) * max(K, 1) ** -0.5).to(BF)
        self.B = (randn(L, N, r) * r ** -0.5).to(BF)
        self.C = randn(T, N)
        self.scale = 0.25 + torch.rand(L, generator=g) if with_scale else None
        self.bias = randn(N) if with_bias else None
        if order == "none":
            self.ids = torch.full((T,), -1, dtype=torch.int32)
        elif order == "one":
            self.ids = torch.full((T,), L - 1, dtype=torch.int32)
        else:
            self.ids = torch.randint(-1, max(L, 1), (T,), generator=g).to(torch.int32)
            if order == "runs":
                self.ids = self.ids.sort().values.roll(T // 3)
                tail = min(T // 8, 30)      # prompts, and behind them sequences of one row
                self.ids[T - tail:] = torch.randint(-1, max(L, 1), (tail,), generator=g).to(torch.int32)
            if T > 3:
                self.ids[T // 2] = L            # outside: no adapter
                self.ids[T // 3] = -2 ** 31
                self.ids[1] = 2 ** 31 - 1
        self.sizes = (T, N, K, r, L)

    def workspace(self, fill=0xA5):
        return torch.full((max(1, dg.dgemm_adapter_workspace_size(*self.sizes)),), fill, dtype=torch.uint8, device=dev())

    def on_gpu(self, *names):
        return [None if getattr(self, n) is None else getattr(self, n).to(dev()) for n in names]

    def project(self, act="none", out=BF, ws=None, D=None, stream=None):
        T, N = self.sizes[:2]
        X, W, A, B, ids, scale, bias = self.on_gpu("X", "W", "A", "B", "ids", "scale", "bias")
        if D is None:
            D = torch.full((T, N // 2 if act == "swiglu" else N), float("nan"), dtype=out, device=dev())
        ws = self.workspace() if ws is None else ws
        dg.dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, bias=bias, act=act, ws=ws, stream=stream)
        assert status_ok(ws, stream)
        return D

    def add(self, act="none", out=BF, c=BF, in_place=False):
        X, A, B, ids, scale, bias = self.on_gpu("X", "A", "B", "ids", "scale", "bias")
        C = None if c is None else self.C.to(c).to(dev())
        D = C if in_place else torch.full(self.sizes[:2], float("nan"), dtype=out, device=dev())
        ws = self.workspace()
        dg.dgemm_adapter_add(X, A, B, ids, D, C=C, scale=scale, bias=bias, act=act, ws=ws)
        assert status_ok(ws)
        return D


def close(got, want):
    value, tol = want
    got = got.cpu().double()
    bad = ~((got - value).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), value[bad][:4].tolist())


SIZES = [(1, 128, 128, 8, 1), (1, 4096, 4096, 16, 8), (2, 130, 72, 8, 3), (3, 1, 8, 8, 2), (15, 257, 136, 24, 4),
         (16, 512, 512, 16, 5), (17, 1000, 1416, 40, 6), (48, 384, 2048, 32, 30), (64, 640, 320, 64, 50), (65, 129, 200, 128, 7),
         (100, 264, 1024, 8, 40), (130, 2049, 64, 16, 9), (256, 300, 520, 72, 3), (300, 1024, 384, 16, 4), (513, 520, 256, 120, 20),
         (1000, 264, 136, 8, 64)]


@pytest.mark.parametrize("T,N,K,r,L", SIZES)
@pytest.mark.parametrize("order,act", [("mixed", "none"), ("runs", "silu"), ("one", "gelu"), ("none", "relu")])
def test_projection(form, T, N, K, r, L, order, act):
    p = Problem(T, N, K, r, L, order=order, with_bias=order != "mixed", with_scale=order != "one")
    out = F32 if T % 2 else BF
    close(p.project(act, out), ref.adapters(p.X, p.A, p.B, p.ids, W=p.W, scale=p.scale, bias=p.bias, act=act, out_dtype=out))


@pytest.mark.parametrize("T,N,K,r,L", [(1, 256, 128, 16, 2), (20, 130, 264, 8, 7), (64, 768, 1024, 64, 20), (70, 2050, 72, 24, 3),
                                       (300, 512, 512, 16, 6), (700, 260, 320, 128, 4)])
@pytest.mark.parametrize("out", [BF, F32])
def test_gated_projection(form, T, N, K, r, L, out):
    p = Problem(T, N, K, r, L, order="runs" if T > 64 else "mixed", with_bias=T % 3 == 1)
    close(p.project("swiglu", out), ref.adapters(p.X, p.A, p.B, p.ids, W=p.W, scale=p.scale, bias=p.bias, act="swiglu", out_dtype=out))


@pytest.mark.parametrize("T,N,K,r,L", SIZES)
@pytest.mark.parametrize("c,out,act", [(BF, BF, "none"), (F32, BF, "silu"), (BF, F32, "gelu"), (None, F32, "none"), (F32, F32, "relu")])
def test_beside_another_product(form, T, N, K, r, L, c, out, act):
    p = Problem(T, N, K, r, L, seed=1, order="runs" if T > 64 else "mixed", with_bias=act == "silu")
    C = None if c is None else p.C.to(c)
    close(p.add(act, out, c), ref.adapters(p.X, p.A, p.B, p.ids, C=C, scale=p.scale, bias=p.bias, act=act, out_dtype=out))


@pytest.mark.parametrize("T,N", [(5, 300), (64, 304), (400, 300), (400, 304), (1100, 712)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(form, T, N, dtype):
    for order in ("mixed", "none", "runs"):
        p = Problem(T, N, 136, 16, 5, order=order)
        got = p.add("none", dtype, dtype, in_place=True)
        close(got, ref.adapters(p.X, p.A, p.B, p.ids, C=p.C.to(dtype), scale=p.scale, out_dtype=dtype))
        untouched = (p.ids < 0) | (p.ids >= 5)
        assert torch.equal(got.cpu()[untouched], p.C.to(dtype)[untouched])       # their rows keep their bits


@pytest.mark.parametrize("T", [3, 70, 300])
def test_no_adapters_at_all_and_no_depth(form, T):
    p = Problem(T, 264, 136, 8, 0, with_bias=True)
    close(p.project("silu"), ref.adapters(p.X, p.A, p.B, p.ids, W=p.W, bias=p.bias, act="silu"))
    close(p.add("none", F32, BF), ref.adapters(p.X, p.A, p.B, p.ids, C=p.C.to(BF), bias=p.bias, out_dtype=F32))
    p = Problem(T, 264, 0, 8, 3, with_bias=True)
    assert torch.equal(p.project("none", F32).cpu(), p.bias.expand(T, 264))
    close(p.add("relu", BF, F32), ref.adapters(p.X, p.A, p.B, p.ids, C=p.C, bias=p.bias, act="relu"))


def test_nothing_to_do():
    p = Problem(0, 64, 64, 8, 2)
    assert p.project().shape == (0, 64)
    p = Problem(4, 0, 64, 8, 2)
    assert p.project().shape == (4, 0) and p.add().shape == (4, 0)


@pytest.mark.parametrize("T,order", [(8, "mixed"), (60, "mixed"), (200, "runs"), (300, "runs"), (520, "mixed")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_adapter_stays_with_its_request(form, T, order, bad):
    p = Problem(T, 264, 256, 16, 6, order=order)
    calls = [(lambda: p.project(out=F32).cpu(), dict(W=p.W), F32), (lambda: p.add(out=F32, c=F32).cpu(), dict(C=p.C), F32),
             (lambda: p.add(out=BF, c=BF).cpu(), dict(C=p.C.to(BF)), BF)]
    clean = [call() for call, _, _ in calls]
    hit = p.ids == 2
    assert bool(hit.any()) and not bool(hit.all())
    for where in ("A", "B"):
        keep = getattr(p, where).clone()
        getattr(p, where)[2, 3, 5] = bad
        for (call, beside, out), was in zip(calls, clean):
            got = call()
            assert torch.equal(got[~hit], was[~hit])
            want = ref.adapters(p.X, p.A, p.B, p.ids, **beside, scale=p.scale, out_dtype=out)[0]
            assert torch.equal(torch.isfinite(got), torch.isfinite(want))
            # one infinite factor: the same infinity (or NaN where infinities of both signs or a NaN meet)
            if where == "B":
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)].to(out))
        setattr(p, where, keep)


@pytest.mark.parametrize("T,K,r", [(256, 256, 16), (400, 64, 32), (300, 128, 24), (520, 64, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_adapter_that_whole_tiles_share(form, T, K, r, bad):
    # V = +-1 and +-1.01 (not a BF16 number): its rest is 0 or has the other sign, and the infinity stays what it is
    p = Problem(T, 264, K, r, 6, order="none")
    p.ids[:] = 2
    p.ids[T // 256 * 256:] = 4
    p.X[:] = 0
    p.X[:, 0] = torch.tensor([1.0, -1.0, 1.0078125, -1.0078125] * T)[:T].to(BF)
    p.A[:] = 0
    p.A[:, :, 0] = 1.0
    p.A[:, r // 2:, 0] = 1.0078125
    p.scale[:] = 1.0
    p.B[2, 5, 3] = p.B[2, 200, r - 1] = bad
    for got, beside, out in ((p.project(out=F32).cpu(), dict(W=p.W), F32), (p.add(out=BF, c=BF).cpu(), dict(C=p.C.to(BF)), BF),
                             (p.add(out=F32, c=BF).cpu(), dict(C=p.C.to(BF)), F32)):
        want = ref.adapters(p.X, p.A, p.B, p.ids, **beside, scale=p.scale, out_dtype=out)[0]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)].to(out))
        assert torch.equal(torch.isfinite(got), torch.isfinite(want))


@pytest.mark.parametrize("T", [8, 64, 300])
def test_a_bad_row_stays_alone(form, T):
    p = Problem(T, 264, 256, 16, 6, order="one")
    clean = p.project(out=F32).cpu()
    p.X[4, 17] = float("nan")
    p.X[5, 0] = float("inf")
    got = p.project(out=F32).cpu()
    rest = torch.ones(T, dtype=torch.bool)
    rest[4] = rest[5] = False
    assert torch.equal(got[rest], clean[rest]) and bool(got[4].isnan().all()) and not bool(torch.isfinite(got[5]).any())


@pytest.mark.parametrize("T,N,K,r,L,order", [(1, 512, 4096, 16, 4, "mixed"), (40, 640, 1024, 32, 9, "mixed"), (700, 520, 512, 16, 5, "runs")])
def test_the_same_bits_every_time_on_another_stream_and_in_a_graph(form, T, N, K, r, L, order):
    p = Problem(T, N, K, r, L, order=order)
    first = p.project()
    second = p.project(ws=p.workspace(0x00))
    stream = torch.cuda.Stream()
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    ws, third, fourth = p.workspace(), torch.empty_like(first), torch.empty_like(first)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        dg.dgemm_adapter_bf16(X, W, A, B, ids, third, scale=scale, ws=ws)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):                     # one call behind another in the same workspace
            dg.dgemm_adapter_bf16(X, W, A, B, ids, fourth, scale=scale, ws=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third) and torch.equal(first, fourth)


def test_inputs_written_just_before_and_after_the_call():
    # the launches of a call overlap each other and the ones around them: X changes from call to call
    p = Problem(16, 512, 2048, 16, 4)
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    ws = p.workspace()
    Xs = [torch.randn(16, 2048, generator=torch.Generator().manual_seed(i)).to(BF).to(dev()) for i in range(6)]
    want, got = [], []
    for x in Xs:
        want.append(dg.dgemm_adapter_bf16(x, W, A, B, ids, torch.empty(16, 512, dtype=BF, device=dev()), scale=scale, ws=ws).clone())
        torch.cuda.synchronize()
    torch.cuda.synchronize()
    X2 = torch.empty_like(X)
    for x in Xs:
        X2.copy_(x)
        D = torch.empty(16, 512, dtype=BF, device=dev())
        got.append(dg.dgemm_adapter_bf16(X2, W, A, B, ids, D, scale=scale, ws=ws))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [8, 600])
def test_waits_are_bounded(form, T):
    p = Problem(T, 512, 1024, 16, 4, order="runs")
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    D, ws = torch.empty(T, 512, dtype=BF, device=dev()), p.workspace()
    want = p.project().clone()
    with dg.overrides(wait_limit_ns=2_000_000, stall_after_loads=1):
        dg.dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, ws=ws)
        torch.cuda.synchronize()
    assert dg.dgemm_query_device_status(ws) != 0
    dg.dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, ws=ws)      # and the next call is right again
    assert dg.dgemm_query_device_status(ws) == 0 and torch.equal(D, want)


def test_calls_on_two_streams_at_once():
    # each with a workspace of its own
    problems = [Problem(T, 776, 512, r, 9, seed=T, order=o) for T, r, o in ((24, 16, "mixed"), (700, 32, "runs"))]
    want = [(p.project(), p.add()) for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    held = []
    torch.cuda.synchronize()
    for _ in range(8):
        for p, s in zip(problems, streams):
            X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
            C = p.C.to(BF).to(dev())
            out = [torch.empty(p.sizes[0], p.sizes[1], dtype=BF, device=dev()) for _ in range(2)]
            ws = p.workspace()
            torch.cuda.current_stream().synchronize()
            with torch.cuda.stream(s):
                dg.dgemm_adapter_bf16(X, W, A, B, ids, out[0], scale=scale, ws=ws)
                dg.dgemm_adapter_add(X, A, B, ids, out[1], C=C, scale=scale, ws=ws)
            held.append((p, out, (X, W, A, B, ids, scale, C, ws)))
    torch.cuda.synchronize()
    for p, out, _ in held:
        a, b = want[problems.index(p)]
        assert torch.equal(out[0], a) and torch.equal(out[1], b)


def test_the_first_call_inside_a_capture():
    """In a process of its own: nothing has been set up when the graph is captured."""
    import os
    import subprocess
    import sys
    code = """
import torch, dense_gemm_persistent_gb300 as dg
BF = torch.bfloat16
mk = lambda *s: (torch.randn(*s, device="cuda") * 0.1).to(BF)
for T, N in ((4, 256), (400, 4096), (400, 4100)):
    X, W, A, B, C = mk(T, 512), mk(N, 512), mk(6, 16, 512), mk(6, N, 16), mk(T, N)
    ids = torch.randint(-1, 6, (T,), dtype=torch.int32, device="cuda")
    D, E = torch.empty_like(C), torch.empty_like(C)
    ws = torch.empty(dg.dgemm_adapter_workspace_size(T, N, 512, 16, 6), dtype=torch.uint8, device="cuda")
    def calls(D, E):
        dg.dgemm_adapter_bf16(X, W, A, B, ids, D, ws=ws)
        dg.dgemm_adapter_add(X, A, B, ids, E, C=C, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(D, E)
    g.replay()
    torch.cuda.synchronize()
    D2, E2 = torch.empty_like(C), torch.empty_like(C)
    calls(D2, E2)
    torch.cuda.synchronize()
    assert torch.equal(D, D2) and torch.equal(E, E2), (T, N)
    assert dg.dgemm_query_device_status(ws) == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("T", [64, 900])
def test_a_workspace_of_exactly_the_size_and_what_lies_behind(form, T):
    p = Problem(T, 520, 264, 24, 12, order="runs")
    X, W, A, B, ids, scale = p.on_gpu("X", "W", "A", "B", "ids", "scale")
    n = dg.dgemm_adapter_workspace_size(*p.sizes)
    room = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=dev())
    D = torch.full((T + 2, 520), 7.0, dtype=BF, device=dev())
    dg.dgemm_adapter_bf16(X, W, A, B, ids, D[1:T + 1], scale=scale, ws=room[:n])
    close(D[1:T + 1], ref.adapters(p.X, p.A, p.B, p.ids, W=p.W, scale=p.scale))
    assert bool((room[n:] == 0x5A).all()) and bool((D[0] == 7).all()) and bool((D[T + 1] == 7).all())
    with pytest.raises(dg.DgemmError):
        dg.dgemm_adapter_bf16(X, W, A, B, ids, D[1:T + 1], scale=scale, ws=room[:n - 1])


@pytest.mark.parametrize("T,N,K,r", [(60, 136, 64, 8), (260, 264, 72, 16), (1100, 200, 128, 32), (700, 136, 64, 72)])
def test_the_most_adapters_and_tables_on_four_bytes(form, T, N, K, r):
    # every row another of 4096: hundreds in a token tile; ids, scale and bias start on any element
    p = Problem(T, N, K, r, 4096, with_bias=True)
    p.ids[4:] = (torch.arange(T - 4, dtype=torch.int32) * 1361 + 7) % 4096
    X, W, A, B, C = p.on_gpu("X", "W", "A", "B", "C")
    shift = lambda t: torch.cat([t[:1], t]).to(dev())[1:]
    ids, scale, bias = shift(p.ids), shift(p.scale), shift(p.bias)
    assert ids.data_ptr() % 16 == 4
    for C_, out in ((None, BF), (C.to(BF), BF), (C, F32)):
        D, ws = torch.empty(T, N, dtype=out, device=dev()), p.workspace()
        if C_ is None:
            dg.dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, bias=bias, act="silu", ws=ws)
        else:
            dg.dgemm_adapter_add(X, A, B, ids, D, C=C_, scale=scale, bias=bias, act="silu", ws=ws)
        assert status_ok(ws)
        beside = dict(W=p.W) if C_ is None else dict(C=C_.cpu())
        close(D, ref.adapters(p.X, p.A, p.B, p.ids, **beside, scale=p.scale, bias=p.bias, act="silu", out_dtype=out))
