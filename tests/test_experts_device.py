"""The binding of the expert and int8 operators refuses operands, workspaces and streams of
another device than the current one: the library launches on the current device. The
devices are stand-ins; nothing is launched."""
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
from dense_gemm_persistent_gb300 import experts

BF, I32, I8 = torch.bfloat16, torch.int32, torch.int8


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


CALLS = {
    "route": (lambda a, kw: dg.dgemm_route(a["logits"], 2, *(a[n] for n in ("ids", "weights", "offsets", "row_token", "slot_row")), **kw),
              dict(logits=z(6, 8), ids=z(6, 2, dtype=I32), weights=z(6, 2), offsets=z(9, dtype=I32), row_token=z(12, dtype=I32),
                   slot_row=z(6, 2, dtype=I32), ws=z(4096, dtype=torch.uint8))),
    "combine": (lambda a, kw: dg.dgemm_combine(a["Y"], a["slot_row"], a["weights"], a["out"], **kw),
                dict(Y=z(12, 16, dtype=BF), slot_row=z(6, 2, dtype=I32), weights=z(6, 2), out=z(6, 16, dtype=BF),
                     add=z(6, 16, dtype=BF))),
    "grouped_bf16": (lambda a, kw: dg.dgemm_grouped_bf16(a["A"], a["B"], a["offsets"], a["D"], **kw),
                     dict(A=z(10, 32, dtype=BF), B=z(3, 24, 32, dtype=BF), offsets=z(4, dtype=I32), D=z(7, 24, dtype=BF),
                          a_rows=z(7, dtype=I32), bias=z(3, 24), ws=z(256, dtype=torch.uint8))),
    "grouped_fp8": (lambda a, kw: dg.dgemm_grouped_fp8_scaled(a["A"], a["B"], a["sa"], a["sb"], a["offsets"], a["D"], **kw),
                    dict(A=z(10, 32, dtype=torch.uint8), B=z(3, 24, 32, dtype=torch.uint8), sa=z(10), sb=z(3, 24),
                         offsets=z(4, dtype=I32), D=z(7, 24), a_rows=z(7, dtype=I32), bias=z(3, 24), ws=z(256, dtype=torch.uint8))),
    "grouped_int8": (lambda a, kw: dg.dgemm_grouped_int8_scaled(a["A"], a["B"], a["sa"], a["sb"], a["offsets"], a["D"], **kw),
                     dict(A=z(10, 32, dtype=I8), B=z(3, 24, 32, dtype=I8), sa=z(10), sb=z(3, 24), offsets=z(4, dtype=I32),
                          D=z(7, 24), a_rows=z(7, dtype=I32), bias=z(3, 24), ws=z(256, dtype=torch.uint8))),
    "quantize": (lambda a, kw: dg.dgemm_int8_quantize(a["X"], a["q"], a["scale"], **kw),
                 dict(X=z(4, 16), q=z(4, 16, dtype=I8), scale=z(4))),
    "int8": (lambda a, kw: dg.dgemm_int8_scaled(a["A"], a["B"], a["sa"], a["sb"], a["D"], beta=1.0, **kw),
             dict(A=z(5, 32, dtype=I8), B=z(24, 32, dtype=I8), sa=z(5), sb=z(24), D=z(5, 24), C=z(5, 24), bias=z(24),
                  ws=z(256, dtype=torch.uint8))),
}
KEYWORDS = ("ws", "add", "a_rows", "bias", "C")


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 0
        return entry


@pytest.fixture
def rec(monkeypatch):
    """Tensors count as CUDA tensors; its places give a tensor's device, its now the current one."""
    r = Recorder()
    r.places, r.now = {}, 0
    monkeypatch.setattr(dg, "load", lambda *a, **k: r)
    monkeypatch.setattr(dg, "_on_device", lambda t: True)
    monkeypatch.setattr(experts, "_device_of", lambda t: r.places.get(id(t), 0), raising=False)
    monkeypatch.setattr(experts, "_current_device", lambda: r.now, raising=False)
    return r


def run(name, stream=0):
    call, args = CALLS[name]
    call(args, dict({k: args[k] for k in KEYWORDS if k in args}, stream=stream))


@pytest.mark.parametrize("name", list(CALLS))
def test_one_device_is_taken(rec, name):
    run(name)
    rec.now = 3
    rec.places = {id(t): 3 for t in CALLS[name][1].values()}
    run(name)
    assert len(rec.calls) == 2


@pytest.mark.parametrize("name,operand", [(n, o) for n, (_, a) in CALLS.items() for o in a])
def test_an_operand_of_another_device_is_refused(rec, name, operand):
    rec.places = {id(CALLS[name][1][operand]): 1}
    with pytest.raises(ValueError, match="cuda:1"):
        run(name)
    assert not rec.calls


@pytest.mark.parametrize("name", list(CALLS))
def test_another_current_device_is_refused(rec, name):
    rec.places = {id(t): 1 for t in CALLS[name][1].values()}
    with pytest.raises(ValueError, match="current device"):
        run(name)
    assert not rec.calls


@pytest.mark.parametrize("name", list(CALLS))
def test_a_stream_of_another_device_is_refused(rec, name, monkeypatch):
    class Stream:
        cuda_stream = 0

        def __init__(self, index):
            self.device_index = index
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    run(name, Stream(0))
    with pytest.raises(ValueError, match="stream"):
        run(name, Stream(1))
    assert len(rec.calls) == 1


def test_c_that_is_not_read_may_live_anywhere(rec):
    a = CALLS["int8"][1]
    rec.places = {id(a["C"]): 1}
    dg.dgemm_int8_scaled(a["A"], a["B"], a["sa"], a["sb"], a["D"], C=a["C"], stream=0)
    assert rec.calls == ["dgemm_int8_scaled"]
