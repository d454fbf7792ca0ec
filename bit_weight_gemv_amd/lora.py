"""Binding of include/q4_lora.h: low-rank adapters beside a packed projection,
forward and backward.  Argument marshalling only.

    Y = q4_gemm_lora(codes, scales, X, A, B, scaling, ids)
    dX, dA, dB = q4_gemm_lora_backward(dY, codes, scales, X, A, B, scaling, ids)
"""
from __future__ import annotations

import ctypes

from . import _base

EXPORTED = ("q4_gemm_lora_ws_bytes", "q4_gemm_lora", "q4_gemm_lora_backward_ws_bytes", "q4_gemm_lora_backward")

Q4_MAX_RANK = 128
Q4_MAX_ADAPTERS = 1024
Q4_MAX_TOKENS = 1 << 22

_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_ARGS = {
    "q4_gemm_lora_ws_bytes": ([_I64] * 5, _SZ),
    "q4_gemm_lora": ([_P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I32, _P, _P, _SZ, _P], _I32),
    "q4_gemm_lora_backward_ws_bytes": ([_I64] * 5, _SZ),
    "q4_gemm_lora_backward": ([_P, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _SZ, _P],
                              _I32),
}


@_base.sizes
def q4_gemm_lora_ws_bytes(M: int, K: int, N: int, r: int, L: int) -> int:
    """Bytes of scratch q4_gemm_lora needs for this shape (0: none)."""
    return int(_base.function("q4_gemm_lora_ws_bytes", _ARGS)(M, K, N, r, L))


@_base.sizes
def q4_gemm_lora_backward_ws_bytes(M: int, K: int, N: int, r: int, L: int) -> int:
    """Bytes of scratch q4_gemm_lora_backward needs for this shape."""
    return int(_base.function("q4_gemm_lora_backward_ws_bytes", _ARGS)(M, K, N, r, L))


def _operands(codes, scales, X, A, B, scaling, ids):
    torch = _base.torch_module()
    if codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("codes must be [M, K/2] and scales [M, K/64]")
    M, K = codes.shape[0], codes.shape[1] * 2
    if scales.shape[0] != M or scales.shape[1] * 64 != K:
        raise ValueError("codes and scales disagree on M, K")
    dev = codes.device
    _base.check(codes, "codes", torch.uint8, dev)
    _base.check(scales, "scales", torch.float16, dev)
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"X must be [N, K={K}]")
    _base.check(X, "X", torch.bfloat16, dev)
    N = X.shape[0]
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [L, r, K] and B [L, M, r]")
    L, r = A.shape[0], A.shape[1]
    if A.shape[2] != K or tuple(B.shape) != (L, M, r):
        raise ValueError(f"A must be [L, r, K={K}] and B [L, M={M}, r]")
    _base.check(A, "A", torch.bfloat16, dev)
    _base.check(B, "B", torch.bfloat16, dev)
    _base.check(scaling, "scaling", torch.float32, dev)
    _base.check(ids, "ids", torch.int32, dev)
    if scaling.numel() != L or ids.numel() != N:
        raise ValueError(f"scaling must have L={L} entries and ids N={N}")
    return M, K, N, r, L, dev


def q4_gemm_lora(codes, scales, X, A, B, scaling, ids, out_dtype=None, Y=None, workspace=None, stream=None):
    """Y[n] = W . X[n] + scaling[a] * B[a] . (A[a] . X[n]) with a = ids[n] (an
    id outside [0, L): no adapter).  codes, scales: a packed M x K matrix; X
    bf16 [N, K], A bf16 [L, r, K], B bf16 [L, M, r], scaling fp32 [L], ids
    int32 [N].  Returns Y [N, M] of out_dtype (bf16 or fp32)."""
    torch = _base.torch_module()
    M, K, N, r, L, dev = _operands(codes, scales, X, A, B, scaling, ids)
    if out_dtype is None:
        out_dtype = Y.dtype if Y is not None else torch.bfloat16
    kind = _base.out_type(out_dtype, "out_dtype")
    with _base.on(dev, stream) as st:
        Y = st.output(Y, (N, M), out_dtype, "Y")
        ws, nb = st.workspace(workspace, q4_gemm_lora_ws_bytes(M, K, N, r, L))
        s = _base.function("q4_gemm_lora", _ARGS)(
            codes.data_ptr(), scales.data_ptr(), M, K, X.data_ptr(), N, A.data_ptr(), B.data_ptr(),
            scaling.data_ptr(), ids.data_ptr(), r, L, kind, Y.data_ptr(), ws, nb, st.handle)
    _base.raise_for(s, "q4_gemm_lora")
    return Y


def q4_gemm_lora_backward(dY, codes, scales, X, A, B, scaling, ids, need_dX=True, need_adapters=True, dX=None,
                          dA=None, dB=None, workspace=None, stream=None):
    """The gradients of q4_gemm_lora for dY bf16 [N, M]: returns (dX bf16
    [N, K], dA fp32 [L, r, K], dB fp32 [L, M, r]), with None in the place of
    what is not asked for.  The packed matrix has no gradient."""
    torch = _base.torch_module()
    M, K, N, r, L, dev = _operands(codes, scales, X, A, B, scaling, ids)
    if tuple(dY.shape) != (N, M):
        raise ValueError(f"dY must be [N={N}, M={M}]")
    _base.check(dY, "dY", torch.bfloat16, dev)
    if not (need_dX or need_adapters):
        raise ValueError("neither dX nor the adapters' gradients are asked for")
    with _base.on(dev, stream) as st:
        dX = st.output(dX, (N, K), torch.bfloat16, "dX") if need_dX else None
        dA = st.output(dA, (L, r, K), torch.float32, "dA") if need_adapters else None
        dB = st.output(dB, (L, M, r), torch.float32, "dB") if need_adapters else None
        ptr = lambda t: t.data_ptr() if t is not None and t.numel() else None  # noqa: E731
        if ptr(dX) is None and ptr(dA) is None:
            return dX, dA, dB
        ws, nb = st.workspace(workspace, q4_gemm_lora_backward_ws_bytes(M, K, N, r, L))
        s = _base.function("q4_gemm_lora_backward", _ARGS)(
            dY.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K, X.data_ptr(), N, A.data_ptr(), B.data_ptr(),
            scaling.data_ptr(), ids.data_ptr(), r, L, ptr(dX), ptr(dA), ptr(dB), ws, nb, st.handle)
    _base.raise_for(s, "q4_gemm_lora_backward")
    return dX, dA, dB
