"""Python binding of include/dgemm_adapters.h: the low-rank adapters of many requests
beside a shared projection.

As in the package's other entry points, the functions only marshal torch tensors to
device pointers and call libdgemm.so; a tensor that the C ABI would misread is refused
before the call.

    dgemm_adapter_bf16(X, W, A, B, ids, D, scale=scale, ws=ws)     # X W^T and the adapters
    dgemm_adapter_add(X, A, B, ids, D, C=Y, scale=scale, ws=ws)    # beside an E4M3 or int8 product Y
"""
from __future__ import annotations

import torch

import dense_gemm_persistent_gb300 as _dg

from ._lib import ACT, F32
from .experts import _BF16, _F32, _FLOATS, _I32, GROUPED_ACT, _act, _device, _float_code, _matrix, _need, _stream, _workspace

_bf16 = torch.bfloat16
_SWIGLU = GROUPED_ACT["swiglu"]


def _low_rank(X, A, B, ids, scale, dev):
    # the common case in few steps; anything else is looked at, and named, below
    if not (X is not None and A is not None and B is not None and X.dtype is _bf16 and A.dtype is _bf16 and B.dtype is _bf16 and X.dim() == 2 and A.dim() == 3 and B.dim() == 3
            and X.is_contiguous() and A.is_contiguous() and B.is_contiguous() and dev >= 0 and A.get_device() == dev
            and B.get_device() == dev):
        _matrix(X, "X", _BF16, dev)
        _matrix(A, "A", _BF16, dev, 3)
        _matrix(B, "B", _BF16, dev, 3)
    T, K = X.shape
    L, r, K2 = A.shape
    L2, N, r2 = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X has K={K}, A has K={K2}")
    if L2 != L or r2 != r:
        raise ValueError(f"A has shape {tuple(A.shape)}, B {tuple(B.shape)}: expected [L,r,K] and [L,N,r]")
    _need(ids, "ids", (T,), _I32, dev)
    if scale is not None:
        _need(scale, "scale", (L,), _F32, dev)
    return T, K, L, r, N


def _tables(ids, scale, bias, T, L, N):
    """The small operands, for _apart."""
    at = lambda t: None if t is None else t.data_ptr()
    return ("ids", at(ids), 4 * T), ("scale", at(scale), 4 * L), ("bias", at(bias), 4 * N)


def _apart(d, d_bytes, *operands):
    """D is written while the operands are still read: (name, address, bytes) of each."""
    end = d + d_bytes
    for name, p, n in operands:
        if p and p < end and d < p + n:
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
    wide = N // 2 if code == _SWIGLU else N
    _need(D, "D", (T, wide), _FLOATS, dev)
    if bias is not None:
        _need(bias, "bias", (N,), _F32, dev)
    x, w, a, b, d, dt = X.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(), D.data_ptr(), _float_code(D)
    work, work_bytes = _workspace(ws, dev)
    _apart(d, T * wide * (4 if dt == F32 else 2), ("X", x, 2 * T * K), ("W", w, 2 * N * K), ("A", a, 2 * L * r * K),
           ("B", b, 2 * L * N * r), ("ws", work, work_bytes), *_tables(ids, scale, bias, T, L, N))
    st = _dg.load().dgemm_adapter_bf16(x, w, a, b, ids.data_ptr(), None if scale is None else scale.data_ptr(), L, r, d, dt, T, N, K,
                                       None if bias is None else bias.data_ptr(), code, work, work_bytes, _stream(stream, dev))
    if st:
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
    if C is not None:
        _need(C, "C", (T, N), _FLOATS, dev)
    if bias is not None:
        _need(bias, "bias", (N,), _F32, dev)
    x, a, b, d, dt = X.data_ptr(), A.data_ptr(), B.data_ptr(), D.data_ptr(), _float_code(D)
    c, ct = (None, F32) if C is None else (C.data_ptr(), _float_code(C))
    work, work_bytes = _workspace(ws, dev)
    _apart(d, T * N * (4 if dt == F32 else 2), ("X", x, 2 * T * K), ("A", a, 2 * L * r * K), ("B", b, 2 * L * N * r),
           ("C", None if c == d and ct == dt else c, T * N * (4 if ct == F32 else 2)), ("ws", work, work_bytes),
           *_tables(ids, scale, bias, T, L, N))
    st = _dg.load().dgemm_adapter_add(x, a, b, ids.data_ptr(), None if scale is None else scale.data_ptr(), L, r, c, ct, d, dt, T,
                                      N, K, None if bias is None else bias.data_ptr(), ACT[act], work, work_bytes,
                                      _stream(stream, dev))
    if st:
        _dg._check(st, "dgemm_adapter_add")
    return D


def dgemm_adapter_workspace_size(T, N, K, r, L) -> int:
    """Workspace bytes that either call needs with these sizes (0 for sizes that are refused)."""
    return int(_dg.load().dgemm_adapter_workspace_size(T, N, K, r, L))
