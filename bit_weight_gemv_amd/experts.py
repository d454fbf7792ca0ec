"""Binding of include/q4_experts.h: routing, products grouped by expert, and
their weighted sum.  Argument marshalling only, as the package's other calls.

    experts, weights, offsets, rows, pos = q4_route_topk(logits, k)
    H = q4_gemm_grouped(gate_codes, gate_scales, X, offsets, rows, up=(up_codes, up_scales))
    Y = q4_gemm_grouped(down_codes, down_scales, H, offsets)
    out = q4_moe_combine(Y, weights, pos)
"""
from __future__ import annotations

import ctypes

from . import _base

EXPORTED = ("q4_route_topk_ws_bytes", "q4_route_topk", "q4_gemm_grouped_ws_bytes", "q4_gemm_grouped",
            "q4_moe_combine")

Q4_MAX_EXPERTS = 1024
Q4_MAX_TOPK = 16
Q4_MAX_SLOTS = 1 << 22
Q4_MAX_ROWS = 1 << 24
Q4_ROUTE_TOPK = 0
Q4_ROUTE_ALL = 1

_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_ARGS = {
    "q4_route_topk_ws_bytes": ([_I64] * 3, _SZ),
    "q4_route_topk": ([_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "q4_gemm_grouped_ws_bytes": ([_I64] * 5 + [_I32], _SZ),
    "q4_gemm_grouped": ([_P] * 4 + [_I64] * 3 + [_P, _I64, _P, _P, _I64, _I32, _P, _P, _SZ, _P], _I32),
    "q4_moe_combine": ([_P, _I32, _I64, _I64, _P, _P, _I64, _I64, _I32, _P, _P], _I32),
}


@_base.sizes
def q4_route_topk_ws_bytes(T: int, E: int, k: int) -> int:
    """Bytes of scratch q4_route_topk needs for this shape (0: none)."""
    return int(_base.function("q4_route_topk_ws_bytes", _ARGS)(T, E, k))


def q4_route_topk(logits, k, mode="topk", experts=None, weights=None, offsets=None, rows=None, pos=None,
                  workspace=None, stream=None):
    """The k experts of each token from logits [T, E] (fp32 or bf16): returns
    (experts int32 [T, k], weights fp32 [T, k], offsets int32 [E + 1], rows
    int32 [T * k], pos int32 [T, k]).  mode "topk": softmax over the chosen
    logits; "all": over all E."""
    torch = _base.torch_module()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if mode not in ("topk", "all"):
        raise ValueError("mode must be 'topk' or 'all'")
    T, E = logits.shape
    dev = logits.device
    kind = _base.out_type(logits.dtype, "logits")
    _base.check(logits, "logits", logits.dtype, dev)
    i32 = torch.int32
    with _base.on(dev, stream) as st:
        experts = st.output(experts, (T, k), i32, "experts")
        weights = st.output(weights, (T, k), torch.float32, "weights")
        offsets = st.output(offsets, (E + 1,), i32, "offsets")
        rows = st.output(rows, (T * k,), i32, "rows")
        pos = st.output(pos, (T, k), i32, "pos")
        need = q4_route_topk_ws_bytes(T, E, k)
        ws, nb = st.workspace(workspace, need)
        r = _base.function("q4_route_topk", _ARGS)(
            logits.data_ptr(), kind, T, E, k, Q4_ROUTE_ALL if mode == "all" else Q4_ROUTE_TOPK, experts.data_ptr(),
            weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(), ws, nb, st.handle)
    _base.raise_for(r, "q4_route_topk")
    return experts, weights, offsets, rows, pos


def _planes(codes, scales, what):
    torch = _base.torch_module()
    if codes.dim() != 3 or scales.dim() != 3:
        raise ValueError(f"{what}: codes must be [E, M, K/2] and scales [E, M, K/64]")
    E, M, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    if tuple(scales.shape[:2]) != (E, M) or scales.shape[2] * 64 != K:
        raise ValueError(f"{what}: codes and scales disagree on E, M, K")
    _base.check(codes, f"{what} codes", torch.uint8, codes.device)
    _base.check(scales, f"{what} scales", torch.float16, codes.device)
    return E, M, K


@_base.sizes
def q4_gemm_grouped_ws_bytes(E: int, M: int, K: int, T: int, R: int, has_up: bool) -> int:
    """Bytes of scratch q4_gemm_grouped needs for this shape (0: none)."""
    return int(_base.function("q4_gemm_grouped_ws_bytes", _ARGS)(E, M, K, T, R, int(bool(has_up))))


def q4_gemm_grouped(codes, scales, X, offsets, rows=None, up=None, out_dtype=None, Y=None, workspace=None,
                    stream=None):
    """Y[p] = W_e . X[rows[p]] for the positions p of each expert e (offsets
    int32 [E + 1]); with up = (codes, scales) of the up matrices, silu(W_e x) *
    (Up_e x).  codes uint8 [E, M, K/2], scales fp16 [E, M, K/64], X bf16
    [T, K], rows int32 [R] or None (position p reads X[p], R = T).  Returns Y
    [R, M] of out_dtype (bf16 or fp32); positions outside every group keep
    what Y held (new outputs are uninitialised there)."""
    torch = _base.torch_module()
    E, M, K = _planes(codes, scales, "gate" if up is not None else "matrix")
    dev = codes.device
    if up is not None and _planes(up[0], up[1], "up") != (E, M, K):
        raise ValueError("the up matrices must have the gate matrices' shape")
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"X must be [T, K={K}]")
    _base.check(X, "X", torch.bfloat16, dev)
    _base.check(offsets, "offsets", torch.int32, dev)
    if offsets.numel() != E + 1:
        raise ValueError(f"offsets must have E + 1 = {E + 1} entries")
    T = X.shape[0]
    R = T
    if rows is not None:
        _base.check(rows, "rows", torch.int32, dev)
        R = rows.numel()
    if up is not None:
        for t, name in zip(up, ("up codes", "up scales")):
            _base.check(t, name, t.dtype, dev)
    if out_dtype is None:
        out_dtype = Y.dtype if Y is not None else torch.bfloat16
    kind = _base.out_type(out_dtype, "out_dtype")
    with _base.on(dev, stream) as st:
        Y = st.output(Y, (R, M), out_dtype, "Y")
        ws, nb = st.workspace(workspace, q4_gemm_grouped_ws_bytes(E, M, K, T, R, up is not None))
        r = _base.function("q4_gemm_grouped", _ARGS)(
            codes.data_ptr(), scales.data_ptr(), up[0].data_ptr() if up is not None else None,
            up[1].data_ptr() if up is not None else None, E, M, K, X.data_ptr(), T, offsets.data_ptr(),
            rows.data_ptr() if rows is not None else None, R, kind, Y.data_ptr(), ws, nb, st.handle)
    _base.raise_for(r, "q4_gemm_grouped")
    return Y


def q4_moe_combine(Y, weights, pos, out_dtype=None, out=None, stream=None):
    """out[t] = sum_s weights[t, s] * Y[pos[t, s]]: Y [R, M] (bf16 or fp32),
    weights fp32 [T, k], pos int32 [T, k]; returns out [T, M] of out_dtype
    (Y's where none is given).  Positions outside [0, R) add nothing."""
    torch = _base.torch_module()
    dev = Y.device
    if Y.dim() != 2 or weights.dim() != 2 or tuple(pos.shape) != tuple(weights.shape):
        raise ValueError("Y must be [R, M], weights and pos [T, k]")
    R, M = Y.shape
    T, k = weights.shape
    y_kind = _base.out_type(Y.dtype, "Y")
    _base.check(Y, "Y", Y.dtype, dev)
    _base.check(weights, "weights", torch.float32, dev)
    _base.check(pos, "pos", torch.int32, dev)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else Y.dtype
    kind = _base.out_type(out_dtype, "out_dtype")
    with _base.on(dev, stream) as st:
        out = st.output(out, (T, M), out_dtype, "out")
        r = _base.function("q4_moe_combine", _ARGS)(Y.data_ptr(), y_kind, R, M, weights.data_ptr(), pos.data_ptr(), T,
                                                    k, kind, out.data_ptr(), st.handle)
    _base.raise_for(r, "q4_moe_combine")
    return out
