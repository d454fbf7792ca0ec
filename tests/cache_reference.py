"""Plain 64-bit forms of the cache's operators (numpy, on the CPU), with the
error that the library's arithmetic allows each output.

Attention.  A score is a sum of D products of q (exact: 8 bits under a power
of two, but for what lies below 2^-24 of the token's largest) and key values
(code - zero) * scale, rounded to fp16 at most (2^-11 of each product's
magnitude), added in fp32; where codes are multiplied first and the zero point
subtracted behind, every step is bounded by 2^-24 of 30 scale |q| each, over
at most D + 16 steps.  With d the largest error of a row's scores, every
softmax weight is within a factor e^(2 d) of its value.  Weights and values
enter the second product as fp16: 2^-11 each, 2^-24 a sum; weights below 2^-24
of the largest may be lost: 2^-24 of the values' magnitudes for each key.

Where codes and zero points are summed apart, out = sum w scale c - sum w scale
zero, each sum has up to 15 scale a weight, rounded by 2^-24 at every one of
(keys + 16) additions: 2^-24 (keys + 16) 30 sum w scale.  A matrix core drops
what lies 2^-24 below the largest product of its 32, aligned as if codes (in
bits 4 to 7 of an fp16) had the smallest normal exponent 2^-14, that is 2^-18
of the largest weight (or q) times one code for every product: 32 2^-18 sum w
scale at most over all keys, and for a score D 2^-18 scale_b max |q|.
"""
import numpy as np


def bf16(v):
    """To bf16 and back, nearest even."""
    v = np.asarray(v, np.float32)
    b = v.view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def values(codes, scales, zeros):
    """codes uint8 [..., D/2], scales and zeros fp16 [..., D/64] -> fp64 [..., D]."""
    x = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    x[..., 0::2] = codes & 15
    x[..., 1::2] = codes >> 4
    rep = lambda a: np.repeat(a.astype(np.float64), 64, axis=-1)  # noqa: E731
    return (x - rep(zeros)) * rep(scales)


def rotate(x, positions, inv_freq, interleaved, amplitude):
    x = np.asarray(x, np.float64).copy()
    half = len(inv_freq)
    a = (np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64))[:, None, :]
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    x1, x2 = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    return x


def pack(x):
    """The rule of q4_pack_affine on fp64 [..., D]: (codes, scales, zeros),
    each decision an exact comparison; blocks that are not finite are NaN."""
    x = np.asarray(x, np.float64)
    x = x.reshape(x.shape[:-1] + (-1, 64))
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[..., None], x, 0.0)
    hi, lo = np.maximum(x.max(-1), 0), np.minimum(x.min(-1), 0)
    with np.errstate(over="ignore"):
        scales = ((hi - lo) / 15).astype(np.float16)
    finite &= np.isfinite(scales)
    s = np.where(finite, scales.astype(np.float64), 0.0)
    half = np.arange(15) + 0.5
    z = ((-lo)[..., None] > half * s[..., None]).sum(-1)
    codes = (x[..., None] > (half - z[..., None])[..., None, :] * s[..., None, None]).sum(-1)
    dead = s == 0
    codes = np.where(dead[..., None], 0, codes).astype(np.uint8)
    z = np.where(dead, 0, z)
    codes = codes.reshape(codes.shape[:-2] + (-1,))
    scales = np.where(finite, scales, np.float16(np.nan)).astype(np.float16)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales, z.astype(np.float16)


def attend(q, cache, table, lens, offsets, causal=True, window=0, scale=None, out_bf16=True):
    """q fp64 [T, Hq, D]; cache: dict of the six planes (numpy); returns
    (out, bound, lse, lse_bound, touched [T])."""
    T, Hq, D = q.shape
    pages, Hkv, page, _ = cache["k_codes"].shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    K = values(cache["k_codes"], cache["k_scales"], cache["k_zeros"])
    V = values(cache["v_codes"], cache["v_scales"], cache["v_zeros"])
    ks, vs = cache["k_scales"].astype(np.float64), cache["v_scales"].astype(np.float64)
    out, bound = np.zeros((T, Hq, D)), np.full((T, Hq, D), 1e-37)
    lse, lse_bound = np.full((T, Hq), -np.inf), np.full((T, Hq), 1e-37)
    touched = np.zeros(T, bool)
    for b in range(len(lens)):
        first, n = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        L = min(max(int(lens[b]), 0), table.shape[1] * page)
        for j in range(n):
            t = first + j
            touched[t] = True
            p = L - n + j
            hi = p + 1 if causal else L
            lo = max(0, p - window + 1) if window else 0
            at = np.arange(lo, max(lo, hi))
            ids = table[b, at // page] if len(at) else np.zeros(0, int)
            ok = (ids >= 0) & (ids < pages)
            at, ids = at[ok], ids[ok]
            if not len(at):
                continue
            k, v, s16 = K[ids, :, at % page], V[ids, :, at % page], ks[ids, :, at % page]  # [m, Hkv, .]
            vs16 = vs[ids, :, at % page]
            for h in range(Hq):
                kh, vh, sh = k[:, h // G], v[:, h // G], s16[:, h // G]
                x = q[t, h]
                s = scale * (kh @ x)
                ax = np.abs(x)
                d = scale * (2.0 ** -11 * (np.abs(kh) @ ax) + (D + 16) * 2.0 ** -24 * 30 * (sh @ ax.reshape(-1, 64).sum(1))
                             + 2.0 ** -24 * ax.max() * np.abs(kh).sum(1) + 64 * 2.0 ** -18 * ax.max() * sh.sum(1)).max() + 2.0 ** -20 * (1 + np.abs(s).max())
                top = s.max()
                e = np.exp(s - top)
                w = e / e.sum()
                lse[t, h] = top + np.log(e.sum())
                lse_bound[t, h] = d + 2.0 ** -22 * abs(lse[t, h]) + 2.0 ** -20
                out[t, h] = w @ vh
                S = w @ np.abs(vh)
                err = (np.expm1(2 * d) + 2.0 ** -10 + (len(at) + 16) * 2.0 ** -24) * S + np.repeat(
                    w @ vs16[:, h // G], 64) * (2.0 ** -24 * (len(at) + 16) * 30 + 2.0 ** -13) + 2.0 ** -24 * w.max() * np.abs(vh).sum(0)
                bound[t, h] += err + (2.0 ** -8 if out_bf16 else 2.0 ** -24) * (np.abs(out[t, h]) + err)
    return out, bound, lse, lse_bound, touched
