"""Host-side checks of the routed-expert and 8-bit integer operators, on the CPU:
exports, argument refusals of the C ABI (before any device call) and of the
Python binding."""
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


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "dgemm_experts.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(dgemm_\w+)\s*\(", text, flags=re.M)))


def test_exports(lib):
    names = declared()
    assert len(names) == 10
    for name in names:
        assert hasattr(lib, name) and name in _lib.SIGNATURES and callable(getattr(dg, name)), name


# ------------------------------------------------------------------ the C ABI

P = 4096   # an aligned non-null address: never read


def route(lib, **o):
    a = dict(logits=P, dt=0, T=8, E=16, k=2, renorm=1, ids=P, weights=P, offsets=P, row_token=P, slot_row=P, ws=P, n=1 << 20)
    a.update(o)
    return lib.dgemm_route(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(dt=2), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(offsets=None), INVALID), (dict(slot_row=None), INVALID),
    (dict(logits=P + 4), MISALIGNED), (dict(ids=P + 2), MISALIGNED), (dict(T=100000, n=64), WORKSPACE),
    (dict(T=100000, ws=None), WORKSPACE)])
def test_route_refusals(lib, over, code):
    assert route(lib, **over) == code


def combine(lib, **o):
    a = dict(Y=P, R=16, slot=P, w=P, add=None, out=P, dt=1, T=8, H=64, k=2)
    a.update(o)
    return lib.dgemm_combine(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(H=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED),
    (dict(dt=2), INVALID), (dict(Y=None), INVALID), (dict(slot=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(Y=P + 2), MISALIGNED), (dict(add=P + 8), MISALIGNED), (dict(out=P + 4), MISALIGNED),
    (dict(T=0), 0), (dict(H=0), 0), (dict(T=1 << 31), UNSUPPORTED)])
def test_combine_refusals(lib, over, code):
    assert combine(lib, **over) == code


def grouped(lib, **o):
    a = dict(A=P, count=32, rows=None, B=P, layout=1, offsets=P, E=4, D=P, dt=1, R=32, N=64, K=128, alpha=1.0, bias=None,
             act=0, ws=None, n=0)
    a.update(o)
    return lib.dgemm_grouped_bf16(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(E=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-8), INVALID), (dict(layout=2), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(act=4, N=63), INVALID), (dict(dt=2), INVALID),
    (dict(count=31), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(D=None), INVALID),
    (dict(offsets=None), INVALID), (dict(E=1025), UNSUPPORTED), (dict(K=1 << 31), UNSUPPORTED),
    (dict(R=1 << 31, count=1 << 31), UNSUPPORTED), (dict(K=100), MISALIGNED), (dict(layout=0, N=60), MISALIGNED),
    (dict(A=P + 8), MISALIGNED), (dict(D=P + 2), MISALIGNED), (dict(offsets=P + 1), MISALIGNED), (dict(ws=P + 8, n=256), MISALIGNED),
    (dict(R=0, count=0), 0), (dict(N=0), 0), (dict(E=0), 0)])
def test_grouped_refusals(lib, over, code):
    assert grouped(lib, **over) == code


def test_scaled_products_refuse_missing_scales(lib):
    for f in (lib.dgemm_grouped_fp8_scaled, lib.dgemm_grouped_int8_scaled):
        assert f(P, 32, None, P, None, P, P, 4, P, 1, 32, 64, 128, 1.0, None, 0, None, 0, None) == INVALID
        assert f(P, 32, None, P, P, None, P, 4, P, 1, 32, 64, 128, 1.0, None, 0, None, 0, None) == INVALID
        assert f(P, 32, None, P, P, P, P, 4, P, 1, 32, 64, 120, 1.0, None, 0, None, 0, None) == MISALIGNED


def int8(lib, **o):
    a = dict(A=P, B=P, sa=P, sb=P, C=None, cdt=0, D=P, dt=1, M=8, N=64, K=128, alpha=1.0, beta=0.0, bias=None, act=0, ws=None, n=0)
    a.update(o)
    return lib.dgemm_int8_scaled(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), INVALID), (dict(K=-16), INVALID), (dict(act=4), INVALID), (dict(dt=2), INVALID), (dict(A=None), INVALID),
    (dict(sa=None), INVALID), (dict(sb=None), INVALID), (dict(beta=1.0), INVALID), (dict(beta=1.0, C=P, cdt=2), INVALID),
    (dict(beta=1.0, C=P + 4), MISALIGNED), (dict(K=100), MISALIGNED), (dict(B=P + 4), MISALIGNED), (dict(sa=P + 2), MISALIGNED),
    (dict(M=0), 0), (dict(N=0), 0)])
def test_int8_refusals(lib, over, code):
    assert int8(lib, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), INVALID), (dict(dt=2), INVALID), (dict(X=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(X=P + 2), MISALIGNED), (dict(q=P + 4), MISALIGNED), (dict(s=P + 1), MISALIGNED), (dict(M=0), 0)])
def test_quantize_refusals(lib, over, code):
    a = dict(X=P, dt=1, q=P, s=P, M=4, K=64)
    a.update(over)
    assert lib.dgemm_int8_quantize(*a.values(), None) == code


def test_workspace_sizes(lib):
    assert dg.dgemm_route_workspace_size(0, 16, 2) == 0
    assert dg.dgemm_route_workspace_size(5000, 64, 8) > 0
    assert dg.dgemm_route_workspace_size(8, 16, 17) == 0
    for kind in ("bf16", "fp8", "int8"):
        assert dg.dgemm_grouped_workspace_size(kind, 64, 8, 256, 512) >= 256
        assert dg.dgemm_grouped_workspace_size(kind, 64, 8, 255, 512, act="swiglu") == 0
    assert dg.dgemm_int8_workspace_size(1, 4096, 4096) >= 256
    assert dg.dgemm_int8_workspace_size(1, 4096, 4097) == 0


# ------------------------------------------------------------------ the binding

class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(dg, "load", lambda *a, **k: r)
    monkeypatch.setattr(dg, "_on_device", lambda t: True)
    return r


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


BF, I32, I8 = torch.bfloat16, torch.int32, torch.int8


def grouped_args(**o):
    a = dict(A=z(10, 32, dtype=BF), B=z(3, 24, 32, dtype=BF), offsets=z(4, dtype=I32), D=z(10, 24, dtype=BF))
    a.update(o)
    return a


def test_grouped_call_passes_sizes(rec):
    a = grouped_args()
    rows = z(20, dtype=I32)
    D = z(20, 12, dtype=BF)
    dg.dgemm_grouped_bf16(a["A"], a["B"], a["offsets"], D, a_rows=rows, act="swiglu", stream=0)
    name, args = rec.calls[-1]
    assert name == "dgemm_grouped_bf16" and args[1] == 10 and args[6] == 3 and args[9:12] == (20, 24, 32) and args[14] == 4
    dg.dgemm_grouped_bf16(a["A"], z(3, 32, 24, dtype=BF), a["offsets"], a["D"], b_layout="kn", stream=0)
    assert rec.calls[-1][1][4] == 0


@pytest.mark.parametrize("over,kw", [
    (dict(A=z(10, 32)), {}), (dict(A=z(10, 40, dtype=BF)), {}), (dict(B=z(24, 32, dtype=BF)), {}),
    (dict(offsets=z(3, dtype=I32)), {}), (dict(offsets=z(4, dtype=torch.int64)), {}), (dict(D=z(9, 24, dtype=BF)), {}),
    (dict(D=z(10, 24, dtype=torch.float16)), {}), (dict(A=z(32, 10, dtype=BF).t()), {}), ({}, dict(act="tanh")),
    ({}, dict(act="swiglu")), ({}, dict(b_layout="nn")), ({}, dict(bias=z(24))), ({}, dict(a_rows=z(10))),
    ({}, dict(a_rows=z(5, 2, dtype=I32)))])
def test_grouped_binding_refusals(rec, over, kw):
    a = grouped_args(**over)
    with pytest.raises(ValueError):
        dg.dgemm_grouped_bf16(a["A"], a["B"], a["offsets"], a["D"], stream=0, **kw)
    assert not rec.calls


def test_scaled_binding_refusals(rec):
    A, B, D, off = z(10, 32, dtype=I8), z(3, 24, 32, dtype=I8), z(10, 24, dtype=BF), z(4, dtype=I32)
    dg.dgemm_grouped_int8_scaled(A, B, z(10), z(3, 24), off, D, stream=0)
    for sa, sb in ((z(9), z(3, 24)), (z(10), z(24)), (None, z(3, 24)), (z(10, dtype=BF), z(3, 24))):
        with pytest.raises(ValueError):
            dg.dgemm_grouped_int8_scaled(A, B, sa, sb, off, D, stream=0)
    with pytest.raises(ValueError):
        dg.dgemm_grouped_fp8_scaled(A, B, z(10), z(3, 24), off, D, stream=0)
    with pytest.raises(ValueError):
        dg.dgemm_int8_scaled(A, B[0], z(10), z(24), D, act="swiglu", stream=0)
    with pytest.raises(ValueError):
        dg.dgemm_int8_scaled(A, B[0], z(10), z(24), D, beta=1.0, stream=0)
    assert len(rec.calls) == 1


def test_route_and_row_binding_refusals(rec):
    ok = dict(ids=z(6, 2, dtype=I32), weights=z(6, 2), offsets=z(9, dtype=I32), row_token=z(12, dtype=I32), slot_row=z(6, 2, dtype=I32))
    x = z(6, 8)
    dg.dgemm_route(x, 2, *ok.values(), stream=0)
    for name, bad in (("ids", z(6, 3, dtype=I32)), ("weights", z(6, 2, dtype=BF)), ("offsets", z(8, dtype=I32)),
                      ("row_token", z(6, 2, dtype=I32)), ("slot_row", None)):
        with pytest.raises(ValueError):
            dg.dgemm_route(x, 2, *{**ok, name: bad}.values(), stream=0)
    with pytest.raises(ValueError):
        dg.dgemm_route(z(6, 8, dtype=torch.float16), 2, *ok.values(), stream=0)
    Y, slot, w, out = z(12, 16, dtype=BF), z(6, 2, dtype=I32), z(6, 2), z(6, 16, dtype=BF)
    dg.dgemm_combine(Y, slot, w, out, stream=0)
    for args, kw in (((z(12, 16), slot, w, out), {}), ((Y, slot, z(6, 3), out), {}), ((Y, slot, w, z(5, 16, dtype=BF)), {}),
                     ((Y, slot, w, out), dict(add=z(6, 16)))):
        with pytest.raises(ValueError):
            dg.dgemm_combine(*args, stream=0, **kw)
    with pytest.raises(ValueError):
        dg.dgemm_int8_quantize(z(4, 8), z(4, 8), z(4), stream=0)
    assert len(rec.calls) == 2


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        dg.dgemm_int8_quantize(z(4, 16), z(4, 16, dtype=I8), z(4), stream=0)
    assert experts.GROUPED_ACT["swiglu"] == 4
