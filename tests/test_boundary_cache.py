"""The entry points of q4_cache.h without a GPU: exported, and bad arguments
refused on the host before any launch.  The pointers are never dereferenced:
each call fails a check first, or has nothing to do."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def q4():
    import bit_weight_gemv_amd as q4
    if not os.path.exists(q4.LIB_PATH):
        from bit_weight_gemv_amd import build
        build.build()
    return q4


def P(i):
    return (i + 1) << 40  # far apart, aligned


def call(name, *args):
    from bit_weight_gemv_amd import _base, cache
    return _base.function(name, cache._ARGS)(*args)


def struct(planes=None, pages=8, heads=2, page=16, D=128):
    from bit_weight_gemv_amd import cache
    return cache.CacheStruct(*(planes or [P(20 + i) for i in range(6)]), pages, heads, page, D)


def test_declared_exported_and_bound(q4):
    from bit_weight_gemv_amd import cache
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4_cache.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(q4_[a-z_0-9]+)\s*\(", text))
    assert names == set(cache.EXPORTED) == set(cache._ARGS)
    for n in names:
        assert hasattr(q4.lib(), n) and hasattr(q4, n)
    for name, value in re.findall(r"#define (Q4_\w+) (\d+)\b", text):
        assert getattr(cache, name) == int(value), name


def append(c=None, k=P(0), v=P(1), kind=1, T=4, ks=256, vs=256, slots=P(2), pos=P(3), freq=P(4), rot=128, q=P(5), qh=4, qs=512,
           qo=P(6)):
    c = struct() if c is None else c
    return call("q4_cache_append", ctypes.addressof(c) if c else None, k, v, kind, T, ks, vs, slots, pos, freq, rot, 0, 1.0, q, qh,
                qs, qo, None)


def read(c=None, slots=P(0), n=4, kind=1, k=P(1), v=P(2)):
    c = struct() if c is None else c
    return call("q4_cache_read", ctypes.addressof(c) if c else None, slots, n, kind, k, v, None)


def attend(c=None, q=P(0), T=4, qh=4, qs=512, table=P(1), B=4, tp=3, lens=P(2), off=P(3), max_q=4, causal=1, window=0, scale=0.1,
           kind=1, out=P(4), lse=P(5), ws=None, nb=0, own_ws=True):
    c = struct() if c is None else c
    if own_ws and ws is None:
        ws, nb = P(9), 1 << 39
    return call("q4_cache_attend", q, T, qh, qs, ctypes.addressof(c) if c else None, table, B, tp, lens, off, max_q, causal, window,
                scale, kind, out, lse, ws, nb, None)


BAD_CACHE = [dict(pages=-1), dict(heads=0), dict(heads=1025), dict(page=8), dict(page=24), dict(page=8192), dict(D=0), dict(D=96),
             dict(D=320), dict(pages=1 << 27, page=16), dict(pages=1 << 62)]


@pytest.mark.parametrize("f", [append, read, attend])
def test_bad_caches(q4, f):
    for kw in BAD_CACHE:
        assert f(c=struct(**kw)) == q4.Q4_ERR_SHAPE, kw
    assert f(c=False) == q4.Q4_ERR_NULL
    for i in range(6):
        p = [P(20 + j) for j in range(6)]
        p[i] = None
        assert f(c=struct(p)) == q4.Q4_ERR_NULL, i
        p[i] = P(20 + i) + 8
        assert f(c=struct(p)) == q4.Q4_ERR_ALIGN, i


def test_append_refusals(q4):
    S, N, A, O = q4.Q4_ERR_SHAPE, q4.Q4_ERR_NULL, q4.Q4_ERR_ALIGN, q4.Q4_ERR_OVERLAP
    for kw in (dict(kind=2), dict(T=-1), dict(T=(1 << 22) + 1), dict(ks=255), dict(ks=260), dict(vs=248), dict(vs=1 << 40),
               dict(rot=-16), dict(rot=8), dict(rot=144), dict(qh=0), dict(qh=1025), dict(qs=511), dict(qs=516)):
        assert append(**kw) == S, kw
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(freq=None), dict(qo=None)):
        assert append(**kw) == N, kw
    for kw in (dict(k=P(0) + 8), dict(v=P(1) + 8), dict(slots=P(2) + 2), dict(pos=P(3) + 2), dict(freq=P(4) + 1), dict(q=P(5) + 8),
               dict(qo=P(6) + 8)):
        assert append(**kw) == A, kw
    plane = 8 * 2 * 16 * 64
    for kw in (dict(k=P(20) + plane - 16), dict(v=P(23)), dict(slots=P(21)), dict(qo=P(5)), dict(qo=P(0) + 2032),
               dict(q=P(0), qo=P(0)), dict(qo=P(24)), dict(c=struct([P(20), P(21), P(22), P(20) + plane - 16, P(24), P(25)]))):
        assert append(**kw) == O, kw
    # Queries, keys and values of one projection's output may lie between each other.
    assert append(T=0, k=None) == q4.Q4_OK
    assert append(T=0, ks=0, vs=0, qs=0) == q4.Q4_OK


def test_read_refusals(q4):
    for kw in (dict(kind=2), dict(n=-1), dict(n=(1 << 22) + 1)):
        assert read(**kw) == q4.Q4_ERR_SHAPE, kw
    assert read(slots=None) == read(k=None, v=None) == q4.Q4_ERR_NULL
    for kw in (dict(slots=P(0) + 1), dict(k=P(1) + 8), dict(v=P(2) + 4)):
        assert read(**kw) == q4.Q4_ERR_ALIGN, kw
    for kw in (dict(k=P(2)), dict(v=P(20)), dict(k=P(0)), dict(k=P(2) + 4 * 2 * 128 * 2 - 16)):
        assert read(**kw) == q4.Q4_ERR_OVERLAP, kw
    assert read(n=0, slots=None, k=None, v=None) == q4.Q4_OK


def test_attend_refusals(q4):
    for kw in (dict(kind=2), dict(T=-1), dict(T=(1 << 22) + 1), dict(B=-1), dict(B=(1 << 22) + 1), dict(qh=3), dict(qh=0),
               dict(qh=1026), dict(qs=511), dict(qs=516), dict(tp=-1), dict(tp=1 << 27), dict(window=-1), dict(window=1 << 31),
               dict(window=5, causal=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(max_q=0), dict(max_q=(1 << 22) + 1), dict(off=None), dict(off=None, max_q=1, T=3)):
        assert attend(**kw) == q4.Q4_ERR_SHAPE, kw
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None)):
        assert attend(**kw) == q4.Q4_ERR_NULL, kw
    for kw in (dict(q=P(0) + 8), dict(table=P(1) + 2), dict(lens=P(2) + 1), dict(off=P(3) + 2), dict(out=P(4) + 8),
               dict(lse=P(5) + 2)):
        assert attend(**kw) == q4.Q4_ERR_ALIGN, kw
    for kw in (dict(out=P(0)), dict(lse=P(2)), dict(lse=P(3)), dict(out=P(20)), dict(lse=P(4) + 4 * 4 * 128 * 2 - 4),
               dict(out=P(1) - 16)):
        assert attend(**kw) == q4.Q4_ERR_OVERLAP, kw
    assert attend(T=0, q=None) == attend(B=0, lens=None) == q4.Q4_OK
    need = q4.q4_cache_attend_ws_bytes(4, 4, 2, 128, 4, 4)
    if need:
        assert attend(ws=P(9), nb=need - 1) == attend(own_ws=False) == q4.Q4_ERR_WORKSPACE
        assert attend(ws=P(9) + 8, nb=need) == q4.Q4_ERR_ALIGN
        assert attend(ws=P(4), nb=need) == attend(ws=P(21), nb=need) == q4.Q4_ERR_OVERLAP
    for bad in ((-1, 4, 2, 128, 4, 4), (4, 3, 2, 128, 4, 4), (4, 4, 2, 100, 4, 4), (4, 4, 2, 128, 4, 0), (0, 4, 2, 128, 4, 4)):
        assert q4.q4_cache_attend_ws_bytes(*bad) == 0


def test_binding_refusals(q4):
    """What the binding refuses before the library is called (CPU tensors)."""
    torch = pytest.importorskip("torch")
    c = q4.q4_cache_new(2, 2, 16, 128, "cpu")
    z = lambda *s, **k: torch.zeros(s, **k)  # noqa: E731
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    k = z(3, 2, 128)
    with pytest.raises(ValueError):
        q4.q4_cache_new(2, 2, 16, 100, "cpu")
    with pytest.raises(TypeError):
        q4.KVCache(c.k_codes, c.k_codes, c.k_zeros, c.v_codes, c.v_scales, c.v_zeros)
    with pytest.raises(ValueError):
        q4.KVCache(c.k_codes, c.k_scales[:1], c.k_zeros, c.v_codes, c.v_scales, c.v_zeros)
    for bad in (lambda: q4.q4_cache_append(c, k, k, z(2, **i32)), lambda: q4.q4_cache_append(c, k, k[:2], z(3, **i32)),
                lambda: q4.q4_cache_append(c, k[:, :1], k[:, :1], z(3, **i32)),
                lambda: q4.q4_cache_append(c, k.transpose(0, 1).contiguous().transpose(0, 1), k, z(3, **i32)),
                lambda: q4.q4_cache_append(c, k, k, z(3, **i32), inv_freq=z(64)),
                lambda: q4.q4_cache_append(c, k, k, z(3, **i32), inv_freq=z(64), positions=z(2, **i32)),
                lambda: q4.q4_cache_append(c, k, k, z(3, **i32), q_out=z(3, 4, 128, **bf)),
                lambda: q4.q4_cache_append(c, k, k, z(3, **i32)),            # not on a GPU
                lambda: q4.q4_cache_attend(z(3, 4, 128, **bf), c, z(2, 2, **i32), z(2, **i32)),
                lambda: q4.q4_cache_attend(z(2, 3, 128, **bf), c, z(2, 2, **i32), z(2, **i32)),
                lambda: q4.q4_cache_attend(z(2, 4, 64, **bf), c, z(2, 2, **i32), z(2, **i32)),
                lambda: q4.q4_cache_attend(z(2, 4, 128, **bf), c, z(2, 2, **i32), z(3, **i32)),
                lambda: q4.q4_cache_attend(z(2, 4, 128, **bf), c, z(2, 2, **i32), z(2, **i32), q_offsets=z(2, **i32))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q4_cache_append(c, k, k.bfloat16(), z(3, **i32)), lambda: q4.q4_cache_append(c, k.half(), k.half(), z(3, **i32)),
                lambda: q4.q4_cache_append(c, k, k, z(3)), lambda: q4.q4_cache_read(c, z(3)),
                lambda: q4.q4_cache_read(c, z(3, **i32), out_dtype=torch.float16),
                lambda: q4.q4_cache_attend(z(2, 4, 128), c, z(2, 2, **i32), z(2, **i32)),
                lambda: q4.q4_cache_attend(z(2, 4, 128, **bf), c, z(2, 2), z(2, **i32))):
        with pytest.raises(TypeError):
            bad()
