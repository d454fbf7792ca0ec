"""Binding of include/q4_cache.h: a paged key/value cache in the affine 4-bit
format.  Argument marshalling only, as the package's other calls.

    cache = q4_cache_new(pages, heads, page, D, device)
    q = q4_cache_append(cache, k, v, slots, positions, inv_freq, q=q)
    out = q4_cache_attend(q, cache, table, lens)
    k, v = q4_cache_read(cache, slots)
"""
from __future__ import annotations

import ctypes

from . import _base

EXPORTED = ("q4_cache_append", "q4_cache_read", "q4_cache_attend_ws_bytes", "q4_cache_attend")

Q4_CACHE_MAX_HEADS = 1024
Q4_CACHE_MAX_TOKENS = 4194304
Q4_CACHE_MAX_KEYS = 1073741824
Q4_CACHE_MAX_ROWS = 536870912
Q4_CACHE_MAX_D = 256
Q4_CACHE_MIN_PAGE = 16
Q4_CACHE_MAX_PAGE = 4096

_P, _I64, _I32, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


class CacheStruct(ctypes.Structure):
    """q4_cache of include/q4_cache.h."""
    _fields_ = [(n, _P) for n in ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales", "v_zeros")] + [
        (n, _I64) for n in ("pages", "heads", "page", "D")]


_ARGS = {
    "q4_cache_append": ([_P, _P, _P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64, _I32, _F, _P, _I64, _I64, _P, _P], _I32),
    "q4_cache_read": ([_P, _P, _I64, _I32, _P, _P, _P], _I32),
    "q4_cache_attend_ws_bytes": ([_I64] * 6, _SZ),
    "q4_cache_attend": ([_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I32, _I64, _F, _I32, _P, _P, _P, _SZ, _P],
                        _I32),
}


class KVCache:
    """The six planes of a cache: codes uint8 [pages, heads, page, D/2], scales
    and zeros fp16 [pages, heads, page, D/64], of keys and of values.  The
    object keeps its tensors alive."""

    __slots__ = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales", "v_zeros", "pages", "heads", "page", "D",
                 "device", "struct", "pointer")

    def __init__(self, k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros):
        torch = _base.torch_module()
        if k_codes.dim() != 4:
            raise ValueError("codes must be [pages, heads, page, D/2]")
        self.pages, self.heads, self.page, half = k_codes.shape
        self.D, self.device = 2 * half, k_codes.device
        if half == 0 or half % 32:
            raise ValueError("D must be a positive multiple of 64")
        for t, name, dtype, last in ((k_codes, "k_codes", torch.uint8, half), (k_scales, "k_scales", torch.float16, half // 32),
                                     (k_zeros, "k_zeros", torch.float16, half // 32), (v_codes, "v_codes", torch.uint8, half),
                                     (v_scales, "v_scales", torch.float16, half // 32),
                                     (v_zeros, "v_zeros", torch.float16, half // 32)):
            _base.check(t, name, dtype, self.device)
            if tuple(t.shape) != (self.pages, self.heads, self.page, last):
                raise ValueError(f"{name} must be {[self.pages, self.heads, self.page, last]}, got {list(t.shape)}")
            setattr(self, name, t)
        self.struct = CacheStruct(*(getattr(self, n).data_ptr() for n, _ in CacheStruct._fields_[:6]), self.pages, self.heads,
                                  self.page, self.D)
        self.pointer = ctypes.addressof(self.struct)


def q4_cache_new(pages: int, heads: int, page: int, D: int, device) -> KVCache:
    """An uninitialised cache of pages * page positions."""
    torch = _base.torch_module()
    if D <= 0 or D % 64:
        raise ValueError("D must be a positive multiple of 64")
    planes = []
    for _ in range(2):
        planes.append(torch.empty((pages, heads, page, D // 2), dtype=torch.uint8, device=device))
        planes += [torch.empty((pages, heads, page, D // 64), dtype=torch.float16, device=device) for _ in range(2)]
    return KVCache(*planes)


def _tokens(t, name, D, dtype, device):
    """Checks [T, heads, D] with contiguous heads; the distance of tokens."""
    if t.dim() != 3 or t.shape[2] != D:
        raise ValueError(f"{name} must be [T, heads, D={D}]")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    T, heads, _ = t.shape
    stride, head, one = t.stride()
    if one != 1 or (heads > 1 and head != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return stride if T > 1 else heads * D


def q4_cache_append(cache, k, v, slots, positions=None, inv_freq=None, interleaved=False, amplitude=1.0, q=None, q_out=None,
                    stream=None):
    """Writes keys and values [T, heads, D] (fp32 or bf16; tokens may be apart,
    as in a view of a projection's output) to the cache's slots int32 [T] (-1:
    skipped).  With inv_freq fp32 [rot/2] and positions int32 [T] the first rot
    dimensions of keys, and of q [T, q_heads, D], turn by position * inv_freq:
    pairs (i, i + rot/2), or neighbours if interleaved; amplitude multiplies
    what is turned.  Returns the rotated q (bf16 [T, q_heads, D]), or None
    where none is given."""
    torch = _base.torch_module()
    dev, D = cache.device, cache.D
    kind = _base.out_type(k.dtype, "k")
    ks, vs = _tokens(k, "k", D, k.dtype, dev), _tokens(v, "v", D, k.dtype, dev)
    T = k.shape[0]
    if k.shape[1] != cache.heads or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"k and v must be [T, {cache.heads}, {D}]")
    _base.check(slots, "slots", torch.int32, dev)
    if slots.numel() != T:
        raise ValueError("slots must have T entries")
    rot = 0
    if inv_freq is not None:
        _base.check(inv_freq, "inv_freq", torch.float32, dev)
        rot = 2 * inv_freq.numel()
    if rot:
        if positions is None:
            raise ValueError("a rotation needs positions")
        _base.check(positions, "positions", torch.int32, dev)
        if positions.numel() != T:
            raise ValueError("positions must have T entries")
    qh = qs = 0
    if q is not None:
        qs, qh = _tokens(q, "q", D, k.dtype, dev), q.shape[1]
        if q.shape[0] != T:
            raise ValueError("q must have T tokens")
    elif q_out is not None:
        raise ValueError("q_out without q")
    with _base.on(dev, stream) as st:
        if q is not None:
            q_out = st.output(q_out, (T, qh, D), torch.bfloat16, "q_out")
        r = _base.function("q4_cache_append", _ARGS)(
            cache.pointer, k.data_ptr(), v.data_ptr(), kind, T, ks, vs, slots.data_ptr(),
            positions.data_ptr() if rot else None, inv_freq.data_ptr() if rot else None, rot, bool(interleaved), amplitude,
            q.data_ptr() if q is not None else None, qh, qs, q_out.data_ptr() if q is not None else None, st.handle)
    _base.raise_for(r, "q4_cache_append")
    return q_out


def q4_cache_read(cache, slots, out_dtype=None, k_out=None, v_out=None, stream=None, keys=True, values=True):
    """(keys, values) [n, heads, D] of the slots int32 [n], in bf16 or fp32;
    a slot outside the cache reads as zeros.  keys or values False: not read,
    and None in its place."""
    torch = _base.torch_module()
    dev = cache.device
    _base.check(slots, "slots", torch.int32, dev)
    n = slots.numel()
    if not (keys or values):
        raise ValueError("neither keys nor values to read")
    if (k_out is not None and not keys) or (v_out is not None and not values):
        raise ValueError("an output of what is not read")
    if out_dtype is None:
        out_dtype = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else torch.bfloat16
    kind = _base.out_type(out_dtype, "out_dtype")
    shape = (n, cache.heads, cache.D)
    with _base.on(dev, stream) as st:
        if keys:
            k_out = st.output(k_out, shape, out_dtype, "k_out")
        if values:
            v_out = st.output(v_out, shape, out_dtype, "v_out")
        r = _base.function("q4_cache_read", _ARGS)(cache.pointer, slots.data_ptr(), n, kind, k_out.data_ptr() if keys else None,
                                                   v_out.data_ptr() if values else None, st.handle)
    _base.raise_for(r, "q4_cache_read")
    return k_out, v_out


@_base.sizes
def q4_cache_attend_ws_bytes(T: int, q_heads: int, heads: int, D: int, B: int, max_q: int) -> int:
    """Bytes of scratch q4_cache_attend needs for this shape (0: none)."""
    return int(_base.function("q4_cache_attend_ws_bytes", _ARGS)(T, q_heads, heads, D, B, max_q))


def q4_cache_attend(q, cache, table, lens, q_offsets=None, max_q=None, causal=True, window=0, scale=None, out_dtype=None,
                    return_lse=False, out=None, lse=None, workspace=None, stream=None):
    """Attention of the tokens q (bf16 [T, q_heads, D]) over the cached keys and
    values of their sequences: table int32 [B, table_pages] (a sequence's pages
    in order), lens int32 [B] (its keys, the new tokens' included), q_offsets
    int32 [B + 1] (its tokens; None: one token each).  max_q: the most new
    tokens that a sequence has (T where none is given).  A token sees the keys
    up to its own position (causal), the last `window` of them if window > 0.
    scale: 1 / sqrt(D) where none is given.  Returns out [T, q_heads, D] (bf16
    or fp32; weights are rounded by 2^-11 for both), with return_lse (out, lse
    fp32 [T, q_heads]); prompts are slower with lse, whose scores are kept in
    fp32's precision.  Single tokens beside longer rows are faster in a call of
    their own."""
    torch = _base.torch_module()
    dev, D = cache.device, cache.D
    qs = _tokens(q, "q", D, torch.bfloat16, dev)
    T, qh, _ = q.shape
    if qh % cache.heads:
        raise ValueError("the heads of q must be a multiple of the cache's")
    _base.check(table, "table", torch.int32, dev)
    _base.check(lens, "lens", torch.int32, dev)
    if table.dim() != 2 or lens.numel() != table.shape[0]:
        raise ValueError("table must be [B, table_pages] and lens [B]")
    B, table_pages = table.shape
    if q_offsets is not None:
        _base.check(q_offsets, "q_offsets", torch.int32, dev)
        if q_offsets.numel() != B + 1:
            raise ValueError(f"q_offsets must have B + 1 = {B + 1} entries")
        if max_q is None:
            max_q = max(T, 1)
    else:
        if T != B:
            raise ValueError("without q_offsets, q must have a token for each sequence")
        if max_q is None:
            max_q = 1
    if scale is None:
        scale = D ** -0.5
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    kind = _base.out_type(out_dtype, "out_dtype")
    with _base.on(dev, stream) as st:
        out = st.output(out, (T, qh, D), out_dtype, "out")
        if return_lse or lse is not None:
            lse = st.output(lse, (T, qh), torch.float32, "lse")
        ws, nb = st.workspace(workspace, q4_cache_attend_ws_bytes(T, qh, cache.heads, D, B, max_q))
        r = _base.function("q4_cache_attend", _ARGS)(
            q.data_ptr(), T, qh, qs, cache.pointer, table.data_ptr(), B, table_pages, lens.data_ptr(),
            q_offsets.data_ptr() if q_offsets is not None else None, max_q, bool(causal), window, scale, kind,
            out.data_ptr(), lse.data_ptr() if lse is not None else None, ws, nb, st.handle)
    _base.raise_for(r, "q4_cache_attend")
    return (out, lse) if return_lse else out
