"""The entry points of q4_experts.h and q4_lora.h without a GPU: exported, and
bad arguments refused on the host before any launch.  The pointers are never
dereferenced: each call fails a check first, or has nothing to do."""
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


@pytest.mark.parametrize("header,module", [("q4_experts.h", "experts"), ("q4_lora.h", "lora")])
def test_declared_exported_and_bound(q4, header, module):
    import importlib
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(q4_[a-z_0-9]+)\s*\(", text))
    m = importlib.import_module("bit_weight_gemv_amd." + module)
    assert names == set(m.EXPORTED) == set(m._ARGS)
    for n in names:
        assert hasattr(q4.lib(), n) and hasattr(q4, n)
    for name, value in re.findall(r"#define (Q4_\w+) (\d+)\b", text):
        assert getattr(m, name) == int(value), name


def P(i):
    return (i + 1) << 40  # far apart, aligned


def _call(q4, module, name, *args):
    from bit_weight_gemv_amd import _base
    import importlib
    return _base.function(name, importlib.import_module("bit_weight_gemv_amd." + module)._ARGS)(*args)


def _route(q4, T=4, E=8, k=2, kind=0, mode=0, p=None, ws=None, nb=0):
    p = p or [P(i) for i in range(6)]
    return _call(q4, "experts", "q4_route_topk", p[0], kind, T, E, k, mode, p[1], p[2], p[3], p[4], p[5], ws, nb, None)


def test_route_refusals(q4):
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(k=17, E=64), dict(kind=2), dict(mode=2),
               dict(T=(1 << 22) + 1, k=1), dict(T=1 << 62)):
        assert _route(q4, **kw) == q4.Q4_ERR_SHAPE, kw
    for i in range(6):
        p = [P(j) for j in range(6)]
        p[i] = None
        assert _route(q4, p=p) == q4.Q4_ERR_NULL, i
        p[i] = P(i) + 2
        assert _route(q4, p=p) == q4.Q4_ERR_ALIGN, i
    p = [P(j) for j in range(6)]
    p[2] = p[1] + 28                    # weights over the last expert
    assert _route(q4, p=p) == q4.Q4_ERR_OVERLAP
    p[2] = p[0] + 124                   # weights over the last logit
    assert _route(q4, p=p) == q4.Q4_ERR_OVERLAP
    need = q4.q4_route_topk_ws_bytes(65, 8, 2)
    assert q4.q4_route_topk_ws_bytes(32, 8, 2) == 0 and need == 3 * 8 * 4
    assert q4.q4_route_topk_ws_bytes(65, 9, 2) == 3 * 12 * 4
    assert _route(q4, T=65) == q4.Q4_ERR_WORKSPACE
    assert _route(q4, T=65, ws=P(9), nb=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _route(q4, T=65, ws=P(9) + 4, nb=need) == q4.Q4_ERR_ALIGN
    assert _route(q4, T=65, ws=P(4), nb=need) == q4.Q4_ERR_OVERLAP
    assert q4.q4_route_topk_ws_bytes(-1, 8, 2) == 0


def _grouped(q4, E=4, M=32, K=128, T=5, R=10, kind=1, p=None, up=False, rows=True, ws=None, nb=0):
    p = p or [P(i) for i in range(8)]
    return _call(q4, "experts", "q4_gemm_grouped", p[0], p[1], p[2] if up else None, p[3] if up else None, E, M, K, p[4],
                 T, p[5], p[6] if rows else None, R, kind, p[7], ws, nb, None)


def test_grouped_refusals(q4):
    for kw in (dict(E=0), dict(E=1025), dict(M=-1), dict(M=(1 << 24) + 1), dict(K=100), dict(K=0), dict(K=131136),
               dict(T=-1), dict(R=-1), dict(R=(1 << 22) + 1), dict(kind=3), dict(M=1 << 24, R=1 << 22)):
        assert _grouped(q4, **kw) == q4.Q4_ERR_SHAPE, kw
    assert _grouped(q4, R=0, p=[None] * 8) == q4.Q4_OK and _grouped(q4, M=0, p=[None] * 8) == q4.Q4_OK
    for i in (0, 1, 3, 4, 5, 7):
        p = [P(j) for j in range(8)]
        p[i] = None
        assert _grouped(q4, p=p, up=True) == q4.Q4_ERR_NULL, i
    for i, off in ((0, 8), (1, 1), (2, 8), (3, 1), (4, 8), (5, 2), (6, 2), (7, 8)):
        p = [P(j) for j in range(8)]
        p[i] += off
        assert _grouped(q4, p=p, up=True) == q4.Q4_ERR_ALIGN, i
    for i, size in ((0, 4 * 32 * 64), (1, 4 * 32 * 2 * 2), (2, 4 * 32 * 64), (3, 4 * 32 * 2 * 2), (4, 5 * 128 * 2),
                    (5, 20), (6, 40)):
        p = [P(j) for j in range(8)]
        p[7] = p[i] + (size - 1) // 16 * 16   # Y over the last bytes
        assert _grouped(q4, p=p, up=True) == q4.Q4_ERR_OVERLAP, i
    # the tile kernel's workspace, and the partial planes of long rows
    assert q4.q4_gemm_grouped_ws_bytes(4, 32, 128, 5, 10, False) == 0
    assert q4.q4_gemm_grouped_ws_bytes(4, 32, 2112, 5, 10, True) == 2 * 2 * 10 * 32 * 4
    assert q4.q4_gemm_grouped_ws_bytes(1, 32, 128, 5, 20, False) >= 20 * 128 * 2 + 20 * 4
    need = q4.q4_gemm_grouped_ws_bytes(1, 32, 128, 500, 2000, False)
    assert need >= 500 * 128 * 2 + 500 * 4 + 32
    kw = dict(E=1, T=500, R=2000)
    assert _grouped(q4, **kw) == q4.Q4_ERR_WORKSPACE
    assert _grouped(q4, ws=P(9), nb=need - 1, **kw) == q4.Q4_ERR_WORKSPACE
    assert _grouped(q4, ws=P(9) + 8, nb=need, **kw) == q4.Q4_ERR_ALIGN
    assert _grouped(q4, ws=P(4) + 1600, nb=need, **kw) == q4.Q4_ERR_OVERLAP


def test_grouped_workspace_without_rows(q4):
    """With no row of X every position reads as zeros; the tile kernel reads a
    row of its workspace for them all the same, so one row is held."""
    with_one = q4.q4_gemm_grouped_ws_bytes(1, 32, 131072 // 2, 1, 2000, False)
    without = q4.q4_gemm_grouped_ws_bytes(1, 32, 131072 // 2, 0, 2000, False)
    assert with_one - without == 16 and without >= 131072


def _combine(q4, R=10, M=16, T=5, k=2, yk=1, ok=1, p=None):
    p = p or [P(i) for i in range(4)]
    return _call(q4, "experts", "q4_moe_combine", p[0], yk, R, M, p[1], p[2], T, k, ok, p[3], None)


def test_combine_refusals(q4):
    for kw in (dict(R=-1), dict(M=-1), dict(T=-1), dict(k=0), dict(k=17), dict(yk=2), dict(ok=-1),
               dict(T=1 << 22, M=1 << 24)):
        assert _combine(q4, **kw) == q4.Q4_ERR_SHAPE, kw
    assert _combine(q4, T=0, p=[None] * 4) == q4.Q4_OK
    for i in range(4):
        p = [P(j) for j in range(4)]
        p[i] = None
        assert _combine(q4, p=p) == q4.Q4_ERR_NULL, i
        p[i] = P(i) + 2
        assert _combine(q4, p=p) == q4.Q4_ERR_ALIGN, i
    for i, size in ((0, 10 * 16 * 2), (1, 40), (2, 40)):
        p = [P(j) for j in range(4)]
        p[3] = p[i] + (size - 1) // 16 * 16
        assert _combine(q4, p=p) == q4.Q4_ERR_OVERLAP, i


def _lora(q4, M=32, K=128, N=5, r=8, L=2, kind=1, p=None, ws=P(20), nb=1 << 30):
    p = p or [P(i) for i in range(8)]
    return _call(q4, "lora", "q4_gemm_lora", p[0], p[1], M, K, p[2], N, p[3], p[4], p[5], p[6], r, L, kind, p[7], ws, nb,
                 None)


def test_lora_refusals(q4):
    for kw in (dict(M=-1), dict(K=96), dict(N=-1), dict(N=(1 << 22) + 1), dict(r=0), dict(r=12), dict(r=136),
               dict(L=-1), dict(L=1025), dict(kind=2)):
        assert _lora(q4, **kw) == q4.Q4_ERR_SHAPE, kw
    assert _lora(q4, N=0, p=[None] * 8, ws=None) == q4.Q4_OK
    for i in range(8):
        p = [P(j) for j in range(8)]
        p[i] = None
        assert _lora(q4, p=p) == q4.Q4_ERR_NULL, i
        p[i] = P(i) + (1 if i == 1 else 2)
        assert _lora(q4, p=p) == q4.Q4_ERR_ALIGN, i
    for i, size in ((0, 32 * 64), (1, 32 * 4), (2, 5 * 256), (3, 2 * 8 * 256), (4, 2 * 32 * 16), (5, 8), (6, 20)):
        p = [P(j) for j in range(8)]
        p[7] = p[i] + (size - 1) // 16 * 16
        assert _lora(q4, p=p) == q4.Q4_ERR_OVERLAP, i
        assert _lora(q4, ws=P(i)) == q4.Q4_ERR_OVERLAP, i
    need = q4.q4_gemm_lora_ws_bytes(32, 128, 5, 8, 2)
    assert need >= 5 * 8 * 4 + 5 * 128 * 2 + 5 * 4   # A x, the converted activations and their exponents
    assert _lora(q4, ws=None) == q4.Q4_ERR_WORKSPACE and _lora(q4, nb=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _lora(q4, ws=P(20) + 8) == q4.Q4_ERR_ALIGN


def _back(q4, M=32, K=128, N=5, r=8, L=2, p=None, ws=P(20), nb=1 << 30):
    p = p or [P(i) for i in range(11)]
    return _call(q4, "lora", "q4_gemm_lora_backward", p[0], p[1], p[2], M, K, p[3], N, p[4], p[5], p[6], p[7], r, L, p[8],
                 p[9], p[10], ws, nb, None)


def test_lora_backward_refusals(q4):
    for kw in (dict(M=0), dict(M=-1), dict(K=96), dict(N=-1), dict(r=12), dict(L=-1), dict(L=1025)):
        assert _back(q4, **kw) == q4.Q4_ERR_SHAPE, kw
    for i in list(range(8)) + [9, 10]:
        p = [P(j) for j in range(11)]
        p[i] = None
        assert _back(q4, p=p) == q4.Q4_ERR_NULL, i
    p = [P(j) for j in range(8)] + [None] * 3
    assert _back(q4, p=p) == q4.Q4_ERR_NULL          # nothing is asked for
    for i in range(11):
        p = [P(j) for j in range(11)]
        p[i] += 1 if i == 2 else 2
        assert _back(q4, p=p) == q4.Q4_ERR_ALIGN, i
    p = [P(j) for j in range(11)]
    p[10] = p[9] + 16
    assert _back(q4, p=p) == q4.Q4_ERR_OVERLAP       # dB over dA
    p[10] = p[0] + 16
    assert _back(q4, p=p) == q4.Q4_ERR_OVERLAP       # dB over dY
    assert q4.q4_gemm_lora_backward_ws_bytes(32, 128, 0, 8, 2) > 0   # the adapters' empty sums
    need = q4.q4_gemm_lora_backward_ws_bytes(32, 128, 5, 8, 2)
    assert need > 0
    assert _back(q4, ws=None) == q4.Q4_ERR_WORKSPACE and _back(q4, nb=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _back(q4, ws=P(9)) == q4.Q4_ERR_OVERLAP
    p = [P(j) for j in range(11)]
    p[8] = None
    assert _back(q4, p=p, L=0, ws=None) == q4.Q4_OK   # gradients of no adapter: nothing to launch


def test_binding_refusals(q4):
    """Types, shapes, contiguity and devices are refused before the library."""
    import torch
    bf, f, h, u8, i32 = torch.bfloat16, torch.float32, torch.float16, torch.uint8, torch.int32
    z = torch.zeros
    codes, scales = z(2, 8, 32, dtype=u8), z(2, 8, 1, dtype=h)
    X, off = z(3, 64, dtype=bf), z(3, dtype=i32)
    with pytest.raises(ValueError, match="GPU"):
        q4.q4_gemm_grouped(codes, scales, X, off)
    with pytest.raises(TypeError):
        q4.q4_gemm_grouped(codes, scales, X.float(), off)
    with pytest.raises(ValueError, match="contiguous"):
        q4.q4_gemm_grouped(codes, scales, z(64, 3, dtype=bf).t(), off)
    with pytest.raises(ValueError, match="offsets"):
        q4.q4_gemm_grouped(codes, scales, X, z(2, dtype=i32))
    with pytest.raises(ValueError, match="up"):
        q4.q4_gemm_grouped(codes, scales, X, off, up=(z(2, 9, 32, dtype=u8), z(2, 9, 1, dtype=h)))
    with pytest.raises(TypeError):
        q4.q4_gemm_grouped(codes, scales, X, off, out_dtype=h)
    with pytest.raises(ValueError, match="mode"):
        q4.q4_route_topk(z(2, 4), 1, "some")
    with pytest.raises(TypeError):
        q4.q4_route_topk(z(2, 4, dtype=h), 1)
    with pytest.raises(ValueError, match="pos"):
        q4.q4_moe_combine(z(4, 8, dtype=bf), z(2, 2), z(2, 1, dtype=i32))
    a, b = z(2, 8, 64, dtype=bf), z(2, 8, 8, dtype=bf)
    ops = (codes[0], scales[0], X, a, b, z(2), z(3, dtype=i32))
    with pytest.raises(ValueError, match="GPU"):
        q4.q4_gemm_lora(*ops)
    with pytest.raises(ValueError, match="ids"):
        q4.q4_gemm_lora(*ops[:6], z(4, dtype=i32))
    with pytest.raises(ValueError, match="A must"):
        q4.q4_gemm_lora(*ops[:3], z(2, 8, 128, dtype=bf), *ops[4:])
    with pytest.raises(ValueError, match="dY"):
        q4.q4_gemm_lora_backward(z(3, 9, dtype=bf), *ops)
    with pytest.raises(ValueError, match="neither"):
        q4.q4_gemm_lora_backward(z(3, 8, dtype=bf), *ops, need_dX=False, need_adapters=False)
