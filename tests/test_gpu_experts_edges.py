"""Calls of the experts' entry points at the borders of their contract
(q4_experts.h), on the GPU, against plain 64-bit forms.  The bounds are those
of tests/ragged_reference.py."""
import numpy as np
import pytest

import ragged_reference as ref
from test_gpu_experts import _dev, _groups, _packed, _within, _x, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _grouped_c(env, codes, scales, up, X, off, rows, R, Y):
    """q4_gemm_grouped by its C entry point: the binding has R = T where rows is None."""
    torch, q4, dev = env
    from bit_weight_gemv_amd import _base, experts
    E, M, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    need = q4.q4_gemm_grouped_ws_bytes(E, M, K, X.shape[0], R, up is not None)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=dev)
    s = _base.function("q4_gemm_grouped", experts._ARGS)(
        codes.data_ptr(), scales.data_ptr(), up[0].data_ptr() if up else None, up[1].data_ptr() if up else None, E, M, K,
        X.data_ptr(), X.shape[0], off.data_ptr(), rows.data_ptr() if rows is not None else None, R, 0, Y.data_ptr(),
        ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert s == 0
    torch.cuda.synchronize()
    return Y


# E, M, K, sizes, T
BEYOND = [
    (8, 33, 128, [1, 0, 1, 0, 0, 1, 0, 1], 2),        # a row at a time
    (16, 70, 192, [2, 3] * 8, 5),                     # chunks of 16 rows
    (4, 40, 2112, [9, 0, 11, 7], 12),                 # the same in two ranges of K
    (4, 33, 192, [6, 5, 4, 5], 9),
    (2, 70, 320, [30, 29], 31),                       # chunks of 32 rows with an up matrix
    (1, 70, 320, [21], 4),
    (2, 130, 192, [1200, 1190], 1500),                # the tile kernel
    (2, 40, 2112, [3000, 100], 64),                   # in runs of K
    (3, 33, 2112, [5, 0, 9], 0),
]


@pytest.mark.parametrize("E,M,K,sizes,T", BEYOND)
@pytest.mark.parametrize("up", [False, True])
def test_grouped_rows_beyond_x_without_an_index(env, E, M, K, sizes, T, up):  # noqa: F811
    """Without rows position p takes X[p]; a position at or past T takes zeros,
    whichever kernel runs."""
    torch, q4, dev = env
    rng = np.random.default_rng(E + M + K + T)
    R = sum(sizes)
    gate, upm = _packed(rng, E, M, K), _packed(rng, E, M, K)
    X = _x(rng, T, K)
    off = _groups(rng, E, sizes)
    Y = torch.full((R, M), -7.0, device=dev)
    _grouped_c(env, _dev(env, gate[0]), _dev(env, gate[1]), tuple(_dev(env, a) for a in upm) if up else None,
               _dev(env, X).to(torch.bfloat16), _dev(env, off), None, R, Y)
    assert torch.all(Y[T:] == 0)
    levels = q4.codebook()
    want, bound = np.zeros((R, M)), np.full((R, M), 1e-37)
    for e in range(E):
        lo, hi = off[e], min(off[e + 1], T)
        if lo >= hi:
            continue
        x = X[lo:hi].astype(np.float64)
        y, b = ref.product(ref.dequantise(levels, gate[0][e], gate[1][e]), gate[1][e], x)
        if up:
            u, bu = ref.product(ref.dequantise(levels, upm[0][e], upm[1][e]), upm[1][e], x)
            y, b = ref.swiglu(y, b, u, bu)
        want[lo:hi], bound[lo:hi] = y, ref.rounded(y, b, False)
    _within(Y, want, bound, f"beyond X: E={E} R={R} T={T}")


def _same_kind(got, want, what):
    """NaN, +infinity and -infinity where the formula has them, finite elsewhere."""
    got = got.float().cpu().numpy()
    for name, f in (("nan", np.isnan), ("inf", np.isposinf), ("-inf", np.isneginf)):
        bad = f(got) != f(want)
        assert not bad.any(), f"{what}: {name} differs at {np.argwhere(bad)[:4].tolist()}"


@pytest.mark.parametrize("E,M,K,sizes", [
    (8, 33, 192, [1, 0, 1, 0, 0, 1, 0, 1]),
    (16, 70, 192, [2, 3] * 8),
    (4, 40, 2112, [9, 0, 11, 7]),
    (1, 70, 320, [21]),
    (1, 70, 64, [40]),
    (2, 130, 192, [1200, 1190]),
    (1, 300, 64, [1100]),
    (2, 40, 2112, [3000, 100]),
    (1, 1030, 192, [8300]),
])
def test_grouped_infinite_activation(env, E, M, K, sizes):  # noqa: F811
    """An infinity in a row, also in its last weights, where a kernel's steps
    reach past the row, gives what the formula gives: infinities, and NaN where
    the weight is 0."""
    torch, q4, dev = env
    rng = np.random.default_rng(M + K)
    R = sum(sizes)
    codes, scales = _packed(rng, E, M, K)
    X = _x(rng, R, K)
    off = _groups(rng, E, sizes)
    at = {0: K - 1, R // 2: K - 33, R - 1: 5}
    for i, k in at.items():
        X[i, k] = np.inf if i else -np.inf
    y = q4.q4_gemm_grouped(_dev(env, codes), _dev(env, scales), _dev(env, X).to(torch.bfloat16), _dev(env, off),
                           out_dtype=torch.float32)
    levels = q4.codebook()
    rows = sorted(at)
    want = np.zeros((len(rows), M))
    for j, i in enumerate(rows):
        e = int(np.searchsorted(off[1:], i, side="right"))
        with np.errstate(invalid="ignore"):
            want[j] = (ref.dequantise(levels, codes[e], scales[e]) * X[i].astype(np.float64)[None, :]).sum(1)
    assert np.isinf(want).any()
    _same_kind(y[torch.tensor(rows, device=dev)], want, f"E={E} M={M} K={K}")
    keep = torch.ones(R, dtype=torch.bool, device=dev)
    keep[torch.tensor(rows, device=dev)] = False
    assert torch.isfinite(y[keep]).all()


def test_combine_of_many_columns(env):  # noqa: F811
    """Tokens times columns past what a column a lane could launch."""
    torch, q4, dev = env
    T, M = 1 << 17, 1 << 15
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    Y = torch.randn((3, M), generator=g, device=dev).to(torch.bfloat16)
    w = torch.rand((T, 1), generator=g, device=dev)
    pos = torch.randint(0, 3, (T, 1), generator=g, device=dev).to(torch.int32)
    out = q4.q4_moe_combine(Y, w, pos)
    for t in (0, 1, 4097, T // 2, T - 2):
        want = (w[t, 0] * Y[pos[t, 0]].float()).to(torch.bfloat16)   # one product: exact in fp32, one rounding
        assert torch.equal(out[t], want), t


@pytest.mark.parametrize("E,M,K,sizes", [
    (1, 5, 131072, [2]), (1, 5, 131072, [20]), (1, 7, 131008, [40]), (2, 3, 131072, [300, 200]), (1, 130, 65600, [600]),
    (1024, 3, 64, None), (1024, 5, 192, "more"),
])
@pytest.mark.parametrize("up", [False, True])
def test_grouped_largest_k_and_e(env, E, M, K, sizes, up):  # noqa: F811
    rng = np.random.default_rng(E + M + K)
    if sizes is None or sizes == "more":
        sizes = rng.integers(0, 4 if sizes is None else 60, E)
    torch, q4, dev = env
    R = int(np.sum(sizes))
    gate, upm = _packed(rng, E, M, K), _packed(rng, E, M, K)
    X = ref.bf16(rng.standard_normal((R, K)).astype(np.float32))
    off = _groups(rng, E, sizes)
    Y = q4.q4_gemm_grouped(_dev(env, gate[0]), _dev(env, gate[1]), _dev(env, X).to(torch.bfloat16), _dev(env, off),
                           up=tuple(_dev(env, a) for a in upm) if up else None, out_dtype=torch.float32)
    levels = q4.codebook()
    want, bound = np.zeros((R, M)), np.zeros((R, M))
    for e in np.flatnonzero(sizes):
        lo, hi = off[e], off[e + 1]
        x = X[lo:hi].astype(np.float64)
        y, b = ref.product(ref.dequantise(levels, gate[0][e], gate[1][e]), gate[1][e], x)
        if up:
            u, bu = ref.product(ref.dequantise(levels, upm[0][e], upm[1][e]), upm[1][e], x)
            y, b = ref.swiglu(y, b, u, bu)
        want[lo:hi], bound[lo:hi] = y, ref.rounded(y, b, False)
    _within(Y, want, bound, f"E={E} M={M} K={K} R={R} up={up}")


@pytest.mark.parametrize("T,E,k", [(1 << 22, 8, 1), (1 << 18, 64, 16), (70000, 1024, 16)])
def test_route_of_the_most_slots(env, T, E, k):  # noqa: F811
    """Against torch's stable sort, which keeps the order of equal logits."""
    torch, q4, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(T + E)
    logits = torch.randn((T, E), generator=g, device=dev).mul_(4).round_().div_(4)   # with ties
    experts, weights, offsets, rows, pos = q4.q4_route_topk(logits, k)
    top, order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(experts, order[:, :k].to(torch.int32))
    flat = experts.reshape(-1).long()
    by = torch.sort(flat, stable=True)[1]
    assert torch.equal(rows.long(), by // k)
    assert torch.equal(pos.reshape(-1)[by].long(), torch.arange(T * k, device=dev))
    assert torch.equal(offsets[1:].long(), torch.bincount(flat, minlength=E).cumsum(0))
    want = torch.softmax(top[:, :k].double(), 1)
    # expf within 2 steps, k sums of positive terms, one division
    assert bool(((weights.double() - want).abs() <= (k + 8) * 2.0 ** -23 * want + 1e-37).all())


@pytest.mark.parametrize("E,R,K", [(8, 8, 192), (4, 60, 2112), (2, 60, 192), (3, 2600, 192), (3, 2600, 2112)])
@pytest.mark.parametrize("up", [False, True])
def test_grouped_offsets_out_of_order_stay_inside(env, E, R, K, up):  # noqa: F811
    """Offsets that decrease or leave 0 .. R give unspecified results, and
    nothing outside Y and the workspace is written."""
    torch, q4, dev = env
    rng = np.random.default_rng(R + E)
    M = 40
    codes, scales = (_dev(env, a) for a in _packed(rng, E, M, K))
    X = _dev(env, _x(rng, R, K)).to(torch.bfloat16)
    need = q4.q4_gemm_grouped_ws_bytes(E, M, K, R, R, up)
    pad = 1 << 16
    for off in ([0] + [R if e % 2 == 0 else 0 for e in range(E)], [R] * (E + 1), [-5] * E + [R + 77],
                list(range(E, -1, -1)), [2 ** 31 - 1, -2 ** 31] * E):
        off = torch.tensor(off[:E + 1], dtype=torch.int32, device=dev)
        ybuf = torch.full((pad + R * M * 4 + pad,), 85, dtype=torch.uint8, device=dev)
        wbuf = torch.full((pad + need + pad,), 85, dtype=torch.uint8, device=dev)
        Y = ybuf[pad:pad + R * M * 4].view(torch.float32).view(R, M)
        q4.q4_gemm_grouped(codes, scales, X, off, up=(codes, scales) if up else None, Y=Y,
                           workspace=wbuf[pad:pad + need] if need else None)
        torch.cuda.synchronize()
        for b, n in ((ybuf, R * M * 4), (wbuf, need)):
            assert bool((b[:pad] == 85).all()) and bool((b[pad + n:] == 85).all())


@pytest.mark.parametrize("T", [1, 40, 700])
def test_layer_captured(env, T):  # noqa: F811
    """The four calls of a layer in one graph, twice with buffers of their own:
    every replay gives the eager result, with other work between."""
    torch, q4, dev = env
    rng = np.random.default_rng(T)
    E, k, K, F = 16, 4, 320, 192
    g, u, d = ([_dev(env, a) for a in _packed(rng, E, m, n)] for m, n in ((F, K), (F, K), (K, F)))
    xs = [_dev(env, _x(rng, T, K)).to(torch.bfloat16) for _ in range(2)]
    ls = [_dev(env, rng.standard_normal((T, E)).astype(np.float32)) for _ in range(2)]

    def layer(x, logits, stream=None):
        _, w, off, rows, pos = q4.q4_route_topk(logits, k, stream=stream)
        H = q4.q4_gemm_grouped(*g, x, off, rows=rows, up=tuple(u), stream=stream)
        return q4.q4_moe_combine(q4.q4_gemm_grouped(*d, H, off, stream=stream), w, pos, stream=stream)

    eager = [layer(x, l) for x, l in zip(xs, ls)]
    side = torch.cuda.Stream()
    graphs = []
    for x, l in zip(xs, ls):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = layer(x, l, side)
        graphs.append((graph, out))
    for rep in range(3):
        for _, out in graphs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, out), e in zip(graphs, eager):
            assert torch.equal(out, e), rep
        assert torch.equal(layer(xs[0], ls[0]), eager[0])
