"""Plain 64-bit forms of the experts' and the adapters' operators, with the
error that the library's arithmetic allows each output (numpy, on the CPU).

A product of the packed format rounds each table entry to fp16 and its product
with the block's scale to fp16 (half a step each: 2^-11 relative, together at
most 2^-10 + 2^-22), and adds K products in fp32 (2^-24 a sum).  Weights and
activations below fp16's normal range under their power of two (2^-29 of the
row's largest at most, with the truncation of the conversion 2^-28) may be
lost: 2^-27 of the largest magnitudes covers both.
"""
import numpy as np


def bf16(v):
    """To bf16 and back, nearest even."""
    v = np.asarray(v, np.float32)
    b = v.view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def dequantise(levels, codes, scales):
    """codes uint8 [..., M, K/2], scales fp16 [..., M, K/64] -> fp64 [..., M, K]."""
    table = np.asarray(levels, np.float32).astype(np.float64)
    w = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    w[..., 0::2] = table[codes & 15]
    w[..., 1::2] = table[codes >> 4]
    return w * np.repeat(scales.astype(np.float64), 64, axis=-1)


def product(W, scales, X):
    """(y, bound) of X [N, K] by W [M, K], both fp64."""
    K = W.shape[1]
    y = X @ W.T
    S = np.abs(X) @ np.abs(W).T
    ax = np.abs(X)
    biggest = ax.max(1, keepdims=True) if X.shape[0] else np.zeros((0, 1))
    lost = biggest * np.abs(W).sum(1)[None, :] + ax.sum(1, keepdims=True) * np.abs(scales.astype(np.float64)).max(1)[None, :]
    return y, (2.0 ** -10 + 2.0 ** -21 + (K + 64) * 2.0 ** -24) * S + 2.0 ** -27 * lost


def rounded(y, bound, out_bf16):
    """The bound after one rounding to the output type."""
    return bound + (2.0 ** -8 if out_bf16 else 2.0 ** -24) * (np.abs(y) + bound) + 1e-37


def swiglu(g, eg, u, eu):
    """silu(g) * u and its bound: |silu'| <= 1.1; 2^-16 for the exponential
    (its argument's rounding, 88 log2(e) 2^-24 at most, and the quotient)."""
    s = g / (1 + np.exp(-g))
    h = s * u
    return h, 1.1 * eg * np.abs(u) + np.abs(s) * eu + 1.1 * eg * eu + 2.0 ** -16 * (np.abs(h) + np.abs(u) * 1.1 * eg)


def route(logits, k, mode):
    """The contract of q4_route_topk, slot by slot."""
    T, E = logits.shape
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    experts = np.zeros((T, k), np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-l[t, e], e))[:k]
        experts[t] = order
        m = l[t, order[0]]
        if m == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            p = np.where(l[t] == m, 1.0, np.exp(l[t] - m))
        p = np.where(np.isnan(p), 0.0, p)
        weights[t] = p[order] / (p[order].sum() if mode == "topk" else p.sum())
    flat = experts.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
    pos = np.empty(T * k, np.int32)
    pos[order] = np.arange(T * k)
    return experts, weights, offsets, (order // k).astype(np.int32), pos.reshape(T, k)


def lora(levels, codes, scales, X, A, B, scaling, ids):
    """(Y, bound)."""
    W = dequantise(levels, codes, scales)
    y, e = product(W, scales, X)
    K, r = W.shape[1], A.shape[1] if A.ndim == 3 else 0
    for n, a in enumerate(ids):
        if 0 <= a < len(A):
            t = A[a] @ X[n]
            et = K * 2.0 ** -24 * (np.abs(A[a]) @ np.abs(X[n])) + 2.0 ** -23 * np.abs(t)
            d = scaling[a] * (B[a] @ t)
            y[n] += d
            e[n] += scaling[a] * (np.abs(B[a]) @ (et + 2.0 ** -16 * np.abs(t))) + (r + 4) * 2.0 ** -24 * scaling[a] * (
                np.abs(B[a]) @ np.abs(t)) + 2.0 ** -24 * np.abs(y[n])
    return y, e


def lora_backward(levels, codes, scales, X, A, B, scaling, ids, dY):
    """((dX, bound), (dA, bound), (dB, bound))."""
    W = dequantise(levels, codes, scales)
    M, K = W.shape
    N, L, r = X.shape[0], A.shape[0], A.shape[1]
    y = dY @ W
    S = np.abs(dY) @ np.abs(W)
    smax = np.abs(scales.astype(np.float64)).max(1)      # a row's largest scale
    weighed = np.abs(dY) * smax[None, :]
    # Powers of two bring every packed row's largest scale to one magnitude;
    # what a row or a token has below 2^-28 of the largest may be lost.
    lost = 4 * weighed.sum(1, keepdims=True) + 2 * weighed.max(1, keepdims=True) * M
    e = (2.0 ** -10 + 2.0 ** -21 + (M + 64) * 2.0 ** -24) * S + 2.0 ** -27 * lost
    dA, dB = np.zeros((L, r, K)), np.zeros((L, M, r))
    eA, eB = np.zeros((L, r, K)), np.zeros((L, M, r))
    for n, a in enumerate(ids):
        if 0 <= a < L:
            u = scaling[a] * (B[a].T @ dY[n])
            eu = scaling[a] * M * 2.0 ** -24 * (np.abs(B[a]).T @ np.abs(dY[n])) + 2.0 ** -23 * np.abs(u)
            t = scaling[a] * (A[a] @ X[n])
            et = scaling[a] * K * 2.0 ** -24 * (np.abs(A[a]) @ np.abs(X[n])) + 2.0 ** -23 * np.abs(t)
            y[n] += u @ A[a]
            e[n] += (eu + (2.0 ** -16 + (r + 4) * 2.0 ** -24) * np.abs(u)) @ np.abs(A[a]) + 2.0 ** -24 * np.abs(y[n])
            dA[a] += np.outer(u, X[n])
            eA[a] += np.outer(eu + (N + 2) * 2.0 ** -24 * np.abs(u), np.abs(X[n]))
            dB[a] += np.outer(dY[n], t)
            eB[a] += np.outer(np.abs(dY[n]), et + (N + 2) * 2.0 ** -24 * np.abs(t))
    return (y, e), (dA, eA), (dB, eB)
