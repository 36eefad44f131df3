"""Host-side checks of the scored routing and the low-rank adapters, on the CPU:
exports, argument refusals of the C ABI (before any device call) and of the Python
binding."""
import ctypes
import os
import re

import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from dense_gemm_persistent_gb300 import _lib, build, experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dg.load()


def test_exports(lib):
    found = []
    for header in ("dgemm_scored.h", "dgemm_adapters.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        found += re.findall(r"^[A-Za-z_][\w \*]*?\b(dgemm_\w+)\s*\(", text, flags=re.M)
    assert sorted(found) == ["dgemm_adapter_add", "dgemm_adapter_bf16", "dgemm_adapter_workspace_size", "dgemm_route_scored"]
    for name in found:
        assert hasattr(lib, name) and name in _lib.SIGNATURES and callable(getattr(dg, name)) and name in dg.__all__, name


P = 4096   # an aligned non-null address: never read


def route(lib, how=(1, 4, 2, 1, 1, 1.0), **o):
    a = dict(logits=P, dt=0, T=8, E=16, k=2, bias=None, how=None if how is None else _lib.Scoring(*how), ids=P, weights=P, offsets=P,
             row_token=P, slot_row=P, ws=P, n=1 << 20)
    a.update(o)
    return lib.dgemm_route_scored(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(dt=2), INVALID),
    (dict(how=None), INVALID), (dict(how=(2, 1, 1, 0, 1, 1.0)), INVALID), (dict(how=(0, 0, 1, 0, 1, 1.0)), INVALID),
    (dict(how=(0, 3, 1, 0, 1, 1.0)), INVALID), (dict(how=(0, 4, 0, 0, 1, 1.0)), INVALID), (dict(how=(0, 4, 5, 0, 1, 1.0)), INVALID),
    (dict(how=(0, 4, 1, 2, 1, 1.0)), INVALID), (dict(how=(0, 64, 1, 0, 1, 1.0), E=128), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(offsets=None), INVALID), (dict(slot_row=None), INVALID),
    (dict(logits=P + 4), MISALIGNED), (dict(bias=P + 2), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(T=100000, n=64), WORKSPACE), (dict(T=100000, ws=None), WORKSPACE)])
def test_route_scored_refusals(lib, over, code):
    assert route(lib, **over) == code


def project(lib, **o):
    a = dict(X=P, W=P, A=P, B=P, ids=P, scale=None, L=4, r=16, D=P, dt=1, T=32, N=64, K=128, bias=None, act=0, ws=P, n=1 << 20)
    a.update(o)
    return lib.dgemm_adapter_bf16(*a.values(), None)


def add(lib, **o):
    a = dict(X=P, A=P, B=P, ids=P, scale=None, L=4, r=16, C=P, cdt=1, D=P, dt=1, T=32, N=64, K=128, bias=None, act=0, ws=P, n=1 << 20)
    a.update(o)
    return lib.dgemm_adapter_add(*a.values(), None)


COMMON = [
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-8), INVALID), (dict(L=-1), INVALID), (dict(r=0), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(dt=2), INVALID), (dict(X=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(D=None), INVALID), (dict(ids=None), INVALID),
    (dict(L=4097), UNSUPPORTED), (dict(r=136), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(K=1 << 31), UNSUPPORTED),
    (dict(r=12), MISALIGNED), (dict(K=100), MISALIGNED), (dict(X=P + 8), MISALIGNED), (dict(A=P + 2), MISALIGNED),
    (dict(B=P + 8), MISALIGNED), (dict(D=P + 2), MISALIGNED), (dict(ids=P + 2), MISALIGNED), (dict(scale=P + 1), MISALIGNED),
    (dict(bias=P + 2), MISALIGNED), (dict(ws=P + 8), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(n=255), WORKSPACE),
    (dict(T=0), 0), (dict(N=0), 0)]


@pytest.mark.parametrize("over,code", COMMON + [(dict(W=None), INVALID), (dict(W=P + 2), MISALIGNED), (dict(act=4, N=63), INVALID)])
def test_projection_refusals(lib, over, code):
    assert project(lib, **over) == code


@pytest.mark.parametrize("over,code", COMMON + [(dict(act=4), INVALID), (dict(cdt=2), INVALID), (dict(C=P + 2), MISALIGNED),
                                                (dict(cdt=0), INVALID)])
def test_add_refusals(lib, over, code):
    assert add(lib, **over) == code     # (cdt=0: C is D, of another type)


def test_workspace_size(lib):
    size = dg.dgemm_adapter_workspace_size
    assert size(0, 64, 64, 8, 2) >= 256 and size(4096, 64, 64, 64, 2) >= 256 + 4096 * 64 * 4
    assert size(-1, 64, 64, 8, 2) == 0 and size(4, 64, 60, 8, 2) == 0 and size(4, 64, 64, 12, 2) == 0
    assert size(4, 64, 64, 256, 2) == 0 and size(4, 64, 64, 8, 5000) == 0


def refuses(text, call, *a, **kw):
    with pytest.raises(ValueError, match=text):
        call(*a, **kw)


def test_binding_refuses_cpu_tensors_and_words():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    refuses("CUDA tensor", dg.dgemm_route_scored, x, 2, i, x[:, :2], i[0], i[0], i)
    h = torch.zeros(4, 8, dtype=torch.bfloat16)
    refuses("CUDA tensor", dg.dgemm_adapter_bf16, h, h, h[None], h[None], i[0], h)
    refuses("CUDA tensor", dg.dgemm_adapter_add, h, h[None], h[None], i[0], h)


class FakeCuda:
    """What the binding looks at of a tensor, said to be on the GPU."""

    def __init__(self, t, ptr=1 << 20):
        self.t, self.ptr = t, ptr
        self.dtype, self.shape, self.is_cuda, self.nbytes, self.device = t.dtype, t.shape, True, t.nbytes, "cuda:0"

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.ptr


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(experts, "_device_of", lambda t: t.get_device())
    monkeypatch.setattr(experts, "_current_device", lambda: 0)
    monkeypatch.setattr(experts, "_current_raw_stream", lambda dev: 0)
    next_ptr = [1 << 20]

    def make(*shape, dtype=torch.bfloat16, ptr=None):
        next_ptr[0] += 1 << 20
        return FakeCuda(torch.zeros(*shape, dtype=dtype), ptr or next_ptr[0])

    return make


def test_binding_refuses_what_the_library_would_misread(lib, fake):
    f, i = torch.float32, torch.int32
    X, W, A, B, ids, D = fake(8, 64), fake(48, 64), fake(3, 16, 64), fake(3, 48, 16), fake(8, dtype=i), fake(8, 48)
    call, add = dg.dgemm_adapter_bf16, dg.dgemm_adapter_add
    refuses("inner dimensions", call, X, W, fake(3, 16, 72), B, ids, D)
    refuses("expected \\[L,r,K\\]", call, X, W, A, fake(2, 48, 16), ids, D)
    refuses("expected \\[L,r,K\\]", call, X, W, A, fake(3, 48, 8), ids, D)
    refuses("W has shape", call, X, fake(40, 64), A, B, ids, D)
    refuses("ids has dtype", call, X, W, A, B, fake(8, dtype=torch.int64), D)
    refuses("ids has shape", call, X, W, A, B, fake(7, dtype=i), D)
    refuses("scale has shape", call, X, W, A, B, ids, D, scale=fake(2, dtype=f))
    refuses("bias has shape", call, X, W, A, B, ids, D, bias=fake(47, dtype=f))
    refuses("D has shape", call, X, W, A, B, ids, D, act="swiglu")
    refuses("act must be", call, X, W, A, B, ids, D, act="tanh")
    refuses("act must be", add, X, A, B, ids, D, act="swiglu")
    refuses("C has shape", add, X, A, B, ids, D, C=fake(8, 47))
    refuses("D overlaps X", call, X, W, A, B, ids, fake(8, 48, ptr=X.ptr + 64))
    refuses("D overlaps W", call, X, W, A, B, ids, fake(8, 48, ptr=W.ptr - 64))
    refuses("D overlaps C", add, X, A, B, ids, D, C=fake(8, 48, ptr=D.ptr + 32))
    refuses("D overlaps C", add, X, A, B, ids, D, C=fake(8, 48, dtype=f, ptr=D.ptr))
    refuses("D overlaps ws", add, X, A, B, ids, D, ws=fake(1 << 16, dtype=torch.uint8, ptr=D.ptr))
    refuses("D overlaps ids", call, X, W, A, B, fake(8, dtype=i, ptr=D.ptr + 16), D)
    refuses("D overlaps scale", add, X, A, B, ids, D, scale=fake(3, dtype=f, ptr=D.ptr + 16))
    refuses("D overlaps bias", add, X, A, B, ids, D, bias=fake(48, dtype=f, ptr=D.ptr - 16))
    x, e = fake(4, 8, dtype=f), fake(4, 2, dtype=f)
    out = (fake(4, 2, dtype=i), e, fake(9, dtype=i), fake(8, dtype=i), fake(4, 2, dtype=i))
    refuses("score must be", dg.dgemm_route_scored, x, 2, *out, score="tanh")
    refuses("group_score must be", dg.dgemm_route_scored, x, 2, *out, group_score="mean")
    refuses("bias has shape", dg.dgemm_route_scored, x, 2, *out, bias=fake(9, dtype=f))
    with pytest.raises(dg.DgemmError):
        dg.dgemm_route_scored(x, 2, *out, groups=3)


@pytest.mark.parametrize("where", ["X", "W", "A", "B", "ids", "D", "C", "scale", "bias", "ws", "logits", "balance", "offsets"])
def test_binding_refuses_operands_of_another_device(lib, fake, where):
    f, i = torch.float32, torch.int32
    t = dict(X=fake(8, 64), W=fake(48, 64), A=fake(3, 16, 64), B=fake(3, 48, 16), ids=fake(8, dtype=i), D=fake(8, 48),
             C=fake(8, 48), scale=fake(3, dtype=f), bias=fake(48, dtype=f), ws=fake(1 << 16, dtype=torch.uint8),
             logits=fake(4, 8, dtype=f), balance=fake(8, dtype=f), offsets=fake(9, dtype=i))
    t[where].get_device = lambda: 1
    rest = dict(scale=t["scale"], bias=t["bias"], ws=t["ws"])
    calls = [lambda: dg.dgemm_adapter_bf16(t["X"], t["W"], t["A"], t["B"], t["ids"], t["D"], **rest),
             lambda: dg.dgemm_adapter_add(t["X"], t["A"], t["B"], t["ids"], t["D"], C=t["C"], **rest)]
    if where in ("logits", "balance", "offsets"):
        calls = [lambda: dg.dgemm_route_scored(t["logits"], 2, fake(4, 2, dtype=i), fake(4, 2, dtype=f), t["offsets"],
                                               fake(8, dtype=i), fake(4, 2, dtype=i), bias=t["balance"])]
    elif where in ("W", "C"):
        calls = calls[:1] if where == "W" else calls[1:]
    for call in calls:
        with pytest.raises(ValueError, match="cuda:1|current device"):
            call()
