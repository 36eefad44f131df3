"""Python binding of include/dgemm_experts.h: routing, products grouped by
expert, and the 8-bit integer product.

As in the package's other entry points, the functions only marshal torch
tensors to device pointers and call libdgemm.so; a tensor that the C ABI would
misread is refused before the call.

    dgemm_route(logits, k, ids, weights, offsets, row_token, slot_row, ws=ws)
    dgemm_grouped_bf16(X, W13, offsets, H, a_rows=row_token, act="swiglu")
    dgemm_grouped_bf16(H, W2, offsets, Y)
    dgemm_combine(Y, slot_row, weights, out)
"""
from __future__ import annotations

import torch

import dense_gemm_persistent_gb300 as _dg

from ._lib import ACT, B_KN, B_NK, BF16, F32, Scoring

GROUPED_ACT = {**ACT, "swiglu": 4}
SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}
GROUPED_TYPE = {"bf16": 0, "fp8": 1, "int8": 2}

_FLOATS = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_BF16 = (torch.bfloat16,)
_CODES8 = (torch.float8_e4m3fn, torch.uint8)
_INT8 = (torch.int8,)
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_device_of = torch.Tensor.get_device   # -1 on the CPU
_NO_DEVICE = -2                        # no tensor's device: every operand is then looked at, and refused, by name


def _device(t, stream) -> int:
    """The device of a call, by its first operand. The library launches on the current device,
    so the operands have to live there (each is compared as it is checked), and so has a
    stream: kernels would otherwise read another GPU's addresses."""
    if t is None or (dev := _device_of(t)) < 0:
        return _NO_DEVICE
    if dev != _current_device():
        raise ValueError(f"operands are on cuda:{dev}, the current device is cuda:{_current_device()}: "
                         "call inside torch.cuda.device(...)")
    if stream is not None and isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the operands are on cuda:{dev}")
    return dev


def _same_device(t, name, dev):
    if dev >= 0 and _device_of(t) != dev:
        raise ValueError(f"{name} is on cuda:{_device_of(t)}, the call's first operand on cuda:{dev}")


def _need(t, name, shape, dtypes, dev):
    # the common case in few steps; anything else is looked at, and named, below
    if (t is not None and t.dtype in dtypes and t.get_device() == dev and (shape is None or t.shape == shape)
            and t.is_contiguous()):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    _dg._require(t, name, shape, dtypes)
    _same_device(t, name, dev)


def _maybe(t, name, shape, dtypes, dev):
    if t is not None:
        _need(t, name, shape, dtypes, dev)


def _stream(stream, dev):
    """The raw stream: the given one, else the current one of the call's device."""
    if stream is None and dev >= 0:
        return _current_raw_stream(dev)
    return _dg._stream(stream)


def _workspace(ws, dev):
    """(pointer, bytes) of the workspace tensor, or of none."""
    if ws is None:
        return None, 0
    if not (ws.get_device() == dev and ws.is_contiguous()):
        _dg._require(ws, "ws")
        _same_device(ws, "ws", dev)
    return ws.data_ptr(), ws.nbytes


def _matrix(t, name, dtypes, dev, dims=2):
    _need(t, name, None, dtypes, dev)
    if t.dim() != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {dims} dimensions")


def _float_code(t) -> int:
    return F32 if t.dtype == torch.float32 else BF16


def _act(act) -> int:
    if act not in GROUPED_ACT:
        raise ValueError(f"act must be one of {sorted(GROUPED_ACT)}, not {act!r}")
    return GROUPED_ACT[act]


def dgemm_route(logits, k, ids, weights, offsets, row_token, slot_row, *, renormalize=True, ws=None, stream=None):
    """Top-k experts of each token and the (token, slot) pairs grouped by expert.

    logits [T,E] fp32 or bf16; outputs ids [T,k] int32, weights [T,k] fp32,
    offsets [E+1] int32 (rows of expert e are offsets[e]..offsets[e+1]), row_token
    [T*k] int32 (the token of each row, -1 beyond the last), slot_row [T,k] int32.
    Equal logits: lowest expert first; -inf and NaN entries are never chosen (id -1,
    weight 0, row -1 where too few remain). renormalize: weights of the chosen
    experts sum to 1, else they are the softmax over all. ws: uint8 workspace of
    at least dgemm_route_workspace_size(T, E, k) bytes.
    """
    dev = _device(logits, stream)
    _matrix(logits, "logits", _FLOATS, dev)
    T, E = logits.shape
    k = int(k)
    _need(ids, "ids", (T, k), _I32, dev)
    _need(weights, "weights", (T, k), _F32, dev)
    _need(offsets, "offsets", (E + 1,), _I32, dev)
    _need(row_token, "row_token", (T * k,), _I32, dev)
    _need(slot_row, "slot_row", (T, k), _I32, dev)
    code = _dg.load().dgemm_route(logits.data_ptr(), _float_code(logits), T, E, k, int(bool(renormalize)), ids.data_ptr(),
                                  weights.data_ptr(), offsets.data_ptr(), row_token.data_ptr(), slot_row.data_ptr(),
                                  *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(code, "dgemm_route")


def dgemm_route_workspace_size(T, E, k) -> int:
    return int(_dg.load().dgemm_route_workspace_size(T, E, int(k)))


def dgemm_route_scored(logits, k, ids, weights, offsets, row_token, slot_row, *, score="sigmoid", bias=None, groups=1,
                       groups_kept=None, group_score="top2", renormalize=True, scale=1.0, ws=None, stream=None):
    """dgemm_route by scores: s = sigmoid or softmax of the logits, c = s + bias.

    The groups_kept groups (of E / groups consecutive experts) of most worth are kept, ranked
    by the largest c of each ("max") or the sum of its two largest ("top2"); of their
    experts the k largest c are chosen. Weights are s at the chosen experts, divided by
    their sum with renormalize, times scale. Equal values: lowest index first. bias [E]
    fp32 or None; an expert whose logit or bias is -inf or NaN is never chosen.
    groups_kept None: all. Outputs and ws as for dgemm_route.
    """
    dev = _device(logits, stream)
    _matrix(logits, "logits", _FLOATS, dev)
    T, E = logits.shape
    k, groups = int(k), int(groups)
    if score not in SCORE:
        raise ValueError(f"score must be one of {sorted(SCORE)}, not {score!r}")
    if group_score not in GROUP_SCORE:
        raise ValueError(f"group_score must be one of {sorted(GROUP_SCORE)}, not {group_score!r}")
    _maybe(bias, "bias", (E,), _F32, dev)
    _need(ids, "ids", (T, k), _I32, dev)
    _need(weights, "weights", (T, k), _F32, dev)
    _need(offsets, "offsets", (E + 1,), _I32, dev)
    _need(row_token, "row_token", (T * k,), _I32, dev)
    _need(slot_row, "slot_row", (T, k), _I32, dev)
    how = Scoring(SCORE[score], groups, groups if groups_kept is None else int(groups_kept), GROUP_SCORE[group_score],
                  int(bool(renormalize)), float(scale))
    code = _dg.load().dgemm_route_scored(logits.data_ptr(), _float_code(logits), T, E, k, _dg._ptr(bias), how,
                                         ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), row_token.data_ptr(),
                                         slot_row.data_ptr(), *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(code, "dgemm_route_scored")


def dgemm_combine(Y, slot_row, weights, out, *, add=None, stream=None):
    """out[t] = add[t] + sum_j weights[t,j] * Y[slot_row[t,j]], in FP32, rounded once.

    Y [R,H] bf16; slot_row [T,k] int32 (rows outside [0,R) add nothing); weights
    [T,k] fp32; add [T,H] bf16 or None; out [T,H] fp32 or bf16. Returns out.
    """
    dev = _device(Y, stream)
    _matrix(Y, "Y", _BF16, dev)
    _matrix(slot_row, "slot_row", _I32, dev)
    R, H = Y.shape
    T, k = slot_row.shape
    _need(weights, "weights", (T, k), _F32, dev)
    _need(out, "out", (T, H), _FLOATS, dev)
    _maybe(add, "add", (T, H), _BF16, dev)
    code = _dg.load().dgemm_combine(Y.data_ptr(), R, slot_row.data_ptr(), weights.data_ptr(), _dg._ptr(add),
                                    out.data_ptr(), _float_code(out), T, H, k, _stream(stream, dev))
    _dg._check(code, "dgemm_combine")
    return out


def _grouped_sizes(A, B, offsets, D, a_rows, b_layout, bias, act, dtypes, dev):
    _matrix(A, "A", dtypes, dev)
    _matrix(B, "B", dtypes, dev, 3)
    if b_layout == "nk":
        E, N, K = B.shape
    elif b_layout == "kn":
        E, K, N = B.shape
    else:
        raise ValueError(f"b_layout must be 'kn' or 'nk', not {b_layout!r}")
    if A.shape[1] != K:
        raise ValueError(f"inner dimensions differ: A has K={A.shape[1]}, B has K={K}")
    count = A.shape[0]
    R = count
    if a_rows is not None:
        _need(a_rows, "a_rows", None, _I32, dev)
        if a_rows.dim() != 1:
            raise ValueError(f"a_rows has shape {tuple(a_rows.shape)}, expected one dimension")
        R = a_rows.shape[0]
    code = _act(act)
    _need(offsets, "offsets", (E + 1,), _I32, dev)
    _need(D, "D", (R, N // 2 if act == "swiglu" else N), _FLOATS, dev)
    _maybe(bias, "bias", (E, N), _F32, dev)
    return E, R, N, K, count, code


def dgemm_grouped_bf16(A, B, offsets, D, *, a_rows=None, b_layout="nk", bias=None, act="none", alpha=1.0, ws=None,
                       stream=None):
    """D[r] = act(alpha * A[a_rows[r]] . op(B_e) + bias[e]) for the rows r of each expert e.

    A [n,K] bf16; a_rows [R] int32 or None (row r of A); B [E,N,K] ("nk") or [E,K,N]
    ("kn") bf16; offsets [E+1] int32 on the device; bias [E,N] fp32; act in
    none/relu/gelu/silu/swiglu; D [R,N] fp32 or bf16 (swiglu: [R,N/2], the
    gate's channels first in B). K is a multiple of 8; N of "kn" weights too, of 16 with
    swiglu. Rows outside every group are not written.
    ws: optional uint8 workspace (dgemm_grouped_workspace_size). Returns D.
    """
    dev = _device(A, stream)
    E, R, N, K, count, code = _grouped_sizes(A, B, offsets, D, a_rows, b_layout, bias, act, _BF16, dev)
    st = _dg.load().dgemm_grouped_bf16(A.data_ptr(), count, _dg._ptr(a_rows), B.data_ptr(),
                                       B_KN if b_layout == "kn" else B_NK, offsets.data_ptr(), E, D.data_ptr(),
                                       _float_code(D), R, N, K, float(alpha), _dg._ptr(bias), code, *_workspace(ws, dev),
                                       _stream(stream, dev))
    _dg._check(st, "dgemm_grouped_bf16")
    return D


def _grouped_scaled(name, dtypes, Aq, Bq, a_scale, b_scale, offsets, D, a_rows, bias, act, alpha, ws, stream):
    dev = _device(Aq, stream)
    E, R, N, K, count, code = _grouped_sizes(Aq, Bq, offsets, D, a_rows, "nk", bias, act, dtypes, dev)
    _need(a_scale, "a_scale", (count,), _F32, dev)
    _need(b_scale, "b_scale", (E, N), _F32, dev)
    st = getattr(_dg.load(), name)(Aq.data_ptr(), count, _dg._ptr(a_rows), Bq.data_ptr(), a_scale.data_ptr(),
                                   b_scale.data_ptr(), offsets.data_ptr(), E, D.data_ptr(), _float_code(D), R, N, K,
                                   float(alpha), _dg._ptr(bias), code, *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(st, name)
    return D


def dgemm_grouped_fp8_scaled(Aq, Bq, a_scale, b_scale, offsets, D, *, a_rows=None, bias=None, act="none", alpha=1.0,
                             ws=None, stream=None):
    """dgemm_grouped_bf16 with E4M3 codes (float8_e4m3fn or uint8): a_scale [n] fp32 per
    row of A, b_scale [E,N] fp32 per expert and channel. Bq [E,N,K]. Returns D."""
    return _grouped_scaled("dgemm_grouped_fp8_scaled", _CODES8, Aq, Bq, a_scale, b_scale, offsets, D, a_rows, bias, act,
                           alpha, ws, stream)


def dgemm_grouped_int8_scaled(Aq, Bq, a_scale, b_scale, offsets, D, *, a_rows=None, bias=None, act="none", alpha=1.0,
                              ws=None, stream=None):
    """dgemm_grouped_bf16 with int8 codes: a_scale [n] fp32 per row of A, b_scale [E,N]
    fp32 per expert and channel. Bq [E,N,K]. Returns D."""
    return _grouped_scaled("dgemm_grouped_int8_scaled", _INT8, Aq, Bq, a_scale, b_scale, offsets, D, a_rows, bias, act,
                           alpha, ws, stream)


def dgemm_grouped_workspace_size(type, R, E, N, K, *, act="none") -> int:
    """Workspace bytes a grouped call can use; type in bf16/fp8/int8."""
    return int(_dg.load().dgemm_grouped_workspace_size(GROUPED_TYPE[type], R, E, N, K, _act(act)))


def dgemm_int8_quantize(X, q, scale, *, stream=None):
    """Per-row int8 codes: scale [M] = max|X[m]| * (1 / 127) in fp32, q [M,K] = X / scale
    rounded to nearest even. X [M,K] bf16 or fp32. Returns (q, scale)."""
    dev = _device(X, stream)
    _matrix(X, "X", _FLOATS, dev)
    M, K = X.shape
    _need(q, "q", (M, K), _INT8, dev)
    _need(scale, "scale", (M,), _F32, dev)
    code = _dg.load().dgemm_int8_quantize(X.data_ptr(), _float_code(X), q.data_ptr(), scale.data_ptr(), M, K,
                                          _stream(stream, dev))
    _dg._check(code, "dgemm_int8_quantize")
    return q, scale


def dgemm_int8_scaled(Aq, Bq, a_scale, b_scale, D, *, C=None, alpha=1.0, beta=0.0, bias=None, act="none", ws=None,
                      stream=None):
    """D = act(alpha * diag(a_scale) (Aq . Bq^T) diag(b_scale) + beta * C + bias), int8 codes.

    Aq [M,K], Bq [N,K] int8; a_scale [M], b_scale [N] fp32; C, D [M,N] fp32 or bf16;
    bias [N] fp32; act in none/relu/gelu/silu. ws: optional uint8 workspace
    (dgemm_int8_workspace_size). Returns D.
    """
    dev = _device(Aq, stream)
    _matrix(Aq, "Aq", _INT8, dev)
    _matrix(Bq, "Bq", _INT8, dev)
    M, K = Aq.shape
    N = Bq.shape[0]
    if Bq.shape[1] != K:
        raise ValueError(f"inner dimensions differ: Aq has K={K}, Bq has K={Bq.shape[1]}")
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}, not {act!r}")
    _need(a_scale, "a_scale", (M,), _F32, dev)
    _need(b_scale, "b_scale", (N,), _F32, dev)
    _need(D, "D", (M, N), _FLOATS, dev)
    if beta != 0.0:   # C is read only then (and may be None otherwise)
        _need(C, "C", (M, N), _FLOATS, dev)
    _maybe(bias, "bias", (N,), _F32, dev)
    code = _dg.load().dgemm_int8_scaled(Aq.data_ptr(), Bq.data_ptr(), a_scale.data_ptr(), b_scale.data_ptr(),
                                        _dg._ptr(C), _float_code(C) if C is not None else F32, D.data_ptr(),
                                        _float_code(D), M, N, K, float(alpha), float(beta), _dg._ptr(bias), ACT[act],
                                        *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(code, "dgemm_int8_scaled")
    return D


def dgemm_int8_workspace_size(M, N, K) -> int:
    return int(_dg.load().dgemm_int8_workspace_size(M, N, K))
