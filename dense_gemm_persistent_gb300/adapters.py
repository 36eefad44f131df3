"""Python binding of include/dgemm_adapters.h: the low-rank adapters of many requests
beside a shared projection.

As in the package's other entry points, the functions only marshal torch tensors to
device pointers and call libdgemm.so; a tensor that the C ABI would misread is refused
before the call.

    dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, ws=ws)     # X W^T and the adapters
    dgemm_adapter_add(X, A, B, ids, D, C=Y, scale=scale, ws=ws)    # beside an E4M3 or int8 product Y
"""
from __future__ import annotations

import dense_gemm_persistent_gb300 as _dg

from ._lib import ACT, F32
from .experts import _BF16, _F32, _FLOATS, _I32, _act, _device, _float_code, _matrix, _maybe, _need, _stream, _workspace


def _low_rank(X, A, B, ids, scale, dev):
    _matrix(X, "X", _BF16, dev)
    _matrix(A, "A", _BF16, dev, 3)
    _matrix(B, "B", _BF16, dev, 3)
    T, K = X.shape
    L, r, K2 = A.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X has K={K}, A has K={K2}")
    if B.shape[0] != L or B.shape[2] != r:
        raise ValueError(f"A has shape {tuple(A.shape)}, B {tuple(B.shape)}: expected [L,r,K] and [L,N,r]")
    _need(ids, "ids", (T,), _I32, dev)
    _maybe(scale, "scale", (L,), _F32, dev)
    return T, K, L, r, B.shape[1]


def _apart(D, **operands):
    """D is written while the operands are still read."""
    lo = D.data_ptr()
    hi = lo + D.nbytes
    for name, t in operands.items():
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + t.nbytes:
            raise ValueError(f"D overlaps {name}")


def dgemm_adapter_bf16(X, W, A, B, ids, D, *, scale=None, bias=None, act="none", ws=None, stream=None):
    """D[t] = act(X[t] W^T + scale[a] (X[t] A[a]^T) B[a]^T + bias), a = ids[t].

    X [T,K], W [N,K], A [L,r,K], B [L,N,r] bf16; ids [T] int32, a value outside
    [0,L) (-1) for a row without an adapter; scale [L] fp32 or None (1); bias [N] fp32; act in
    none/relu/gelu/silu/swiglu; D [T,N] fp32 or bf16 (swiglu: [T,N/2], the gate's
    channels first in W, B and bias). r (8 to 128) and K are multiples of 8. ws: uint8
    workspace of at least dgemm_adapter_workspace_size(T, N, K, r, L) bytes, for one call
    at a time. Returns D.
    """
    dev = _device(X, stream)
    T, K, L, r, N = _low_rank(X, A, B, ids, scale, dev)
    _need(W, "W", (N, K), _BF16, dev)
    code = _act(act)
    _need(D, "D", (T, N // 2 if act == "swiglu" else N), _FLOATS, dev)
    _maybe(bias, "bias", (N,), _F32, dev)
    _apart(D, X=X, W=W, A=A, B=B, ws=ws)
    st = _dg.load().dgemm_adapter_bf16(X.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(), ids.data_ptr(),
                                       _dg._ptr(scale), L, r, D.data_ptr(), _float_code(D), T, N, K, _dg._ptr(bias), code,
                                       *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(st, "dgemm_adapter_bf16")
    return D


def dgemm_adapter_add(X, A, B, ids, D, *, C=None, scale=None, bias=None, act="none", ws=None, stream=None):
    """D[t] = act(C[t] + scale[a] (X[t] A[a]^T) B[a]^T + bias), a = ids[t].

    C [T,N] fp32 or bf16, the product of another entry point, or None (zero); it may be D
    itself. act in none/relu/gelu/silu. The rest as for dgemm_adapter_bf16. Returns D.
    """
    dev = _device(X, stream)
    T, K, L, r, N = _low_rank(X, A, B, ids, scale, dev)
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}, not {act!r}")
    _need(D, "D", (T, N), _FLOATS, dev)
    _maybe(C, "C", (T, N), _FLOATS, dev)
    _maybe(bias, "bias", (N,), _F32, dev)
    same = C is not None and C.data_ptr() == D.data_ptr() and C.dtype == D.dtype
    _apart(D, X=X, A=A, B=B, C=None if same else C, ws=ws)
    st = _dg.load().dgemm_adapter_add(X.data_ptr(), A.data_ptr(), B.data_ptr(), ids.data_ptr(), _dg._ptr(scale), L, r,
                                      _dg._ptr(C), F32 if C is None else _float_code(C), D.data_ptr(), _float_code(D), T, N,
                                      K, _dg._ptr(bias), ACT[act], *_workspace(ws, dev), _stream(stream, dev))
    _dg._check(st, "dgemm_adapter_add")
    return D


def dgemm_adapter_workspace_size(T, N, K, r, L) -> int:
    """Workspace bytes that either call needs with these sizes (0 for sizes that are refused)."""
    return int(_dg.load().dgemm_adapter_workspace_size(T, N, K, r, L))
