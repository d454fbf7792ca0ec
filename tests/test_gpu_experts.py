"""The experts' operators on the GPU (q4_experts.h) against plain 64-bit forms.
The bounds are those of tests/ragged_reference.py."""
import numpy as np
import pytest

import ragged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible: SKIP (not a pass)")
    import bit_weight_gemv_amd as q4
    q4.lib()
    return torch, q4, torch.device("cuda:0")


def _packed(rng, E, M, K, small=False):
    codes = rng.integers(0, 256, (E, M, K // 2), dtype=np.uint8)
    scales = rng.uniform(0.02, 0.08, (E, M, K // 64))
    if small:  # scales over fp16's whole range, subnormal ones and zero among them
        scales = scales * 2.0 ** rng.integers(-24, 8, (E, M, 1)) * 2.0 ** rng.integers(-6, 1, scales.shape)
        scales[:, ::7] = 0
    return codes, scales.astype(np.float16)


def _dev(env, a):
    torch, _, dev = env
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _x(rng, N, K):
    return ref.bf16(rng.standard_normal((N, K)).astype(np.float32) * rng.choice([0.01, 1.0, 30.0], (N, 1)))


def _within(got, want, bound, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    bad = np.abs(got - want) / np.maximum(bound, 1e-300)
    print(f"{what}: worst |err|/bound = {bad.max() if bad.size else 0:.3g}", flush=True)
    assert np.all(np.abs(got - want) <= bound), f"{what}: worst {bad.max()}"


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------

ROUTES = [(1, 8, 1), (1, 64, 8), (3, 5, 5), (63, 16, 2), (64, 60, 4), (65, 128, 8), (129, 100, 6), (300, 257, 16),
          (1000, 1024, 3), (20000, 64, 8), (2, 1, 1)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("mode", ["topk", "all"])
def test_route(env, T, E, k, mode):
    torch, q4, dev = env
    rng = np.random.default_rng(T * 1000 + E * 10 + k)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    logits[::3] = np.round(logits[::3])            # ties
    got = q4.q4_route_topk(_dev(env, logits), k, mode)
    want = ref.route(logits, k, mode) if T <= 1000 else None
    if want is None:                               # the plain form is slow: the order alone, by numpy
        ex = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
        flat = ex.reshape(-1)
        order = np.argsort(flat, kind="stable")
        pos = np.empty(T * k, np.int32)
        pos[order] = np.arange(T * k)
        l = logits.astype(np.float64)
        p = np.exp(np.take_along_axis(l, ex.astype(np.int64), 1) - l.max(1, keepdims=True))
        w = p / (p.sum(1, keepdims=True) if mode == "topk" else np.exp(l - l.max(1, keepdims=True)).sum(1, keepdims=True))
        off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
        want = ex, w, off, (order // k).astype(np.int32), pos.reshape(T, k)
    for i in (0, 2, 3, 4):
        assert np.array_equal(got[i].cpu().numpy(), want[i]), i
    # expf within 2 steps, up to E sums of positive terms, one division
    bound = (E + 8) * 2.0 ** -23 * want[1] + 1e-37
    assert np.all(np.abs(got[1].cpu().numpy() - want[1]) <= bound)


def test_route_special_values(env):
    torch, q4, dev = env
    inf, nan = np.inf, np.nan
    logits = np.array([[nan, 1, nan, 2], [-inf, -inf, -inf, -inf], [nan, nan, nan, nan], [inf, 0, inf, -inf],
                       [-0.0, 0.0, -0.0, 0.0], [-inf, 5, -inf, -inf],
                       [np.finfo(np.float32).min] * 4, [np.finfo(np.float32).max, 0, -1, 1e-45]], np.float32)
    for mode in ("topk", "all"):
        for k in (1, 2, 4):
            got = q4.q4_route_topk(_dev(env, logits), k, mode)
            want = ref.route(logits, k, mode)
            for i in (0, 2, 3, 4):
                assert np.array_equal(got[i].cpu().numpy(), want[i]), (mode, k, i)
            assert np.allclose(got[1].cpu().numpy(), want[1], rtol=2e-6, atol=1e-37), (mode, k)


def test_route_bf16_and_empty(env):
    torch, q4, dev = env
    rng = np.random.default_rng(5)
    logits = ref.bf16(rng.standard_normal((77, 40)).astype(np.float32))
    a = q4.q4_route_topk(_dev(env, logits).to(torch.bfloat16), 4)
    b = q4.q4_route_topk(_dev(env, logits), 4)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    e = q4.q4_route_topk(torch.empty((0, 40), device=dev), 4)
    assert torch.equal(e[2], torch.zeros(41, dtype=torch.int32, device=dev)) and e[3].numel() == 0


# ---------------------------------------------------------------------------
# Grouped products
# ---------------------------------------------------------------------------

def _groups(rng, E, sizes):
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(sizes)
    return off


def _grouped_case(env, E, M, K, sizes, T, up, gather, out_bf16, seed, small=False, tail=0):
    torch, q4, dev = env
    rng = np.random.default_rng(seed)
    R = int(np.sum(sizes))
    gate, up_m = _packed(rng, E, M, K, small), _packed(rng, E, M, K, small)
    if not gather:
        T = R + tail
    X = _x(rng, T, K)
    off = _groups(rng, E, sizes)
    rows = rng.integers(0, T, R + tail).astype(np.int32) if gather else None
    dt = torch.bfloat16 if out_bf16 else torch.float32
    Y = torch.full((R + tail, M), -7.0, dtype=dt, device=dev)
    q4.q4_gemm_grouped(_dev(env, gate[0]), _dev(env, gate[1]), _dev(env, X).to(torch.bfloat16), _dev(env, off),
                       rows=_dev(env, rows) if gather else None,
                       up=(_dev(env, up_m[0]), _dev(env, up_m[1])) if up else None, Y=Y)
    torch.cuda.synchronize()
    levels = q4.codebook()
    want, bound = np.zeros((R, M)), np.zeros((R, M))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        x = X[rows[lo:hi] if gather else slice(lo, hi)].astype(np.float64)
        y, b = ref.product(ref.dequantise(levels, gate[0][e], gate[1][e]), gate[1][e], x)
        if up:
            u, bu = ref.product(ref.dequantise(levels, up_m[0][e], up_m[1][e]), up_m[1][e], x)
            y, b = ref.swiglu(y, b, u, bu)
        want[lo:hi], bound[lo:hi] = y, ref.rounded(y, b, out_bf16)
    _within(Y[:R], want, bound, f"grouped E={E} M={M} K={K} R={R} up={up}")
    assert torch.all(Y[R:] == -7.0), "rows behind the last group were written"


GROUPED = [
    # E, M, K, sizes, T
    (1, 1, 64, [1], 1),
    (4, 33, 128, [1, 0, 2, 1], 3),
    (8, 70, 192, [0, 0, 0, 8, 0, 0, 0, 0], 5),
    (3, 96, 1408, [9, 8, 7], 11),
    (5, 65, 2048, [33, 0, 1, 32, 31], 20),
    (2, 40, 2112, [5, 1], 4),             # two ranges of K
    (2, 31, 4160, [40, 3], 9),            # three ranges, two chunks
    (66, 17, 64, [1] * 66, 10),           # more experts than lanes
    (2, 300, 256, [130, 129], 200),       # many chunks a group
    (3, 129, 448, [200, 0, 70], 64),
    (1, 520, 128, [257], 300),
    (4, 257, 320, [513, 1, 0, 600], 333),
    (2, 128, 2112, [100, 90], 100),
    (2, 5500, 128, [150, 200], 90),       # tile kernel, 128 rows a piece
    (1, 129, 448, [1100], 300),
    (3, 40, 2112, [1500, 0, 1300], 64),
    (2, 40, 2112, [3000, 100], 64),       # tile kernel, eight runs of K
    (1, 300, 512, [1200], 100),           # one run
    (1, 1030, 64, [8300], 2000),          # 256 rows a piece
    (2, 700, 192, [6100, 6300], 500),
]


@pytest.mark.parametrize("E,M,K,sizes,T", GROUPED)
@pytest.mark.parametrize("up", [False, True])
def test_grouped(env, E, M, K, sizes, T, up):
    for gather in (True, False):
        for out_bf16 in (True, False):
            _grouped_case(env, E, M, K, sizes, T, up, gather, out_bf16, seed=E * 100 + M + K, tail=3)


@pytest.mark.parametrize("sizes", [[3, 1], [150, 140], [1100, 1200]])
def test_grouped_scales_of_every_magnitude(env, sizes):
    _grouped_case(env, 2, 66, 512, sizes, 64, False, True, False, seed=11, small=True)


def test_grouped_rows_outside_and_values_that_are_not_finite(env):
    """A row index outside [0, T) reads as zeros; an infinity or a NaN in one
    activation row leaves every other row's outputs as they were."""
    torch, q4, dev = env
    rng = np.random.default_rng(3)
    for sizes in ([4, 5], [200, 190], [1100, 1050]):
        E, M, K, T = 2, 50, 256, 30
        R = sum(sizes)
        codes, scales = _packed(rng, E, M, K)
        X = _x(rng, T, K)
        off = _groups(rng, E, sizes)
        rows = rng.integers(0, T, R).astype(np.int32)
        rows[1], rows[R - 1] = -1, T
        args = lambda x: (_dev(env, codes), _dev(env, scales), _dev(env, x).to(torch.bfloat16), _dev(env, off))  # noqa: E731
        y0 = q4.q4_gemm_grouped(*args(X), rows=_dev(env, rows), out_dtype=torch.float32)
        assert torch.all(y0[1] == 0) and torch.all(y0[R - 1] == 0)
        bad = X.copy()
        bad[7, 3], bad[8, 5] = np.inf, np.nan
        y1 = q4.q4_gemm_grouped(*args(bad), rows=_dev(env, rows), out_dtype=torch.float32)
        keep = torch.from_numpy((rows != 7) & (rows != 8)).to(dev)
        assert torch.equal(y0[keep], y1[keep])
        if (~keep).any():
            assert not torch.isfinite(y1[~keep]).all()
        z = np.zeros_like(X)
        z[2] = 2.0 ** -126   # the smallest normal value alone in its row
        y2 = q4.q4_gemm_grouped(*args(z), rows=_dev(env, rows), out_dtype=torch.float32)
        assert torch.isfinite(y2).all()


@pytest.mark.parametrize("R", [2, 3, 20, 300, 2200])
def test_grouped_without_rows(env, R):
    """No row of X at all: every index is outside, every output is zero."""
    torch, q4, dev = env
    rng = np.random.default_rng(4)
    codes, scales = (_dev(env, a) for a in _packed(rng, 2, 40, 4160))
    off = _dev(env, _groups(rng, 2, [R // 2, R - R // 2]))
    rows = torch.zeros(R, dtype=torch.int32, device=dev)
    X = torch.empty((0, 4160), dtype=torch.bfloat16, device=dev)
    for up in (None, (codes, scales)):
        y = q4.q4_gemm_grouped(codes, scales, X, off, rows=rows, up=up, out_dtype=torch.float32)
        assert torch.all(y == 0)


def test_grouped_on_another_stream_and_captured(env):
    """The same bits from a call on a side stream, and from a captured call
    replayed with other work in between; two graphs with workspaces of their
    own do not meet."""
    torch, q4, dev = env
    rng = np.random.default_rng(8)
    for sizes, K in (([3, 5], 2112), ([120, 140], 256), ([1100, 1040], 256)):
        E, M, R = 2, 200, sum(sizes)
        codes, scales = (_dev(env, a) for a in _packed(rng, E, M, K))
        off = _dev(env, _groups(rng, E, sizes))
        xs = [_dev(env, _x(rng, R, K)).to(torch.bfloat16) for _ in range(2)]
        eager = [q4.q4_gemm_grouped(codes, scales, x, off) for x in xs]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        y = q4.q4_gemm_grouped(codes, scales, xs[0], off, stream=side)
        side.synchronize()
        assert torch.equal(y, eager[0])
        need = q4.q4_gemm_grouped_ws_bytes(E, M, K, R, R, False)
        graphs = []
        for x in xs:
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
            out = torch.full_like(eager[0], float("nan"))
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=side):
                q4.q4_gemm_grouped(codes, scales, x, off, Y=out, workspace=ws, stream=side)
            graphs.append((g, out, ws))
        for rep in range(3):
            for g, out, _ in graphs:
                out.fill_(float("nan"))
            torch.cuda.synchronize()
            for g, _, _ in graphs:
                g.replay()
            torch.cuda.synchronize()
            for (g, out, _), e in zip(graphs, eager):
                assert torch.equal(out, e), rep
            assert torch.equal(q4.q4_gemm_grouped(codes, scales, xs[0], off), eager[0])


# ---------------------------------------------------------------------------
# Weighted sum
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,M", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 16, 4099), (64, 4, 264), (7, 6, 2056)])
def test_combine(env, T, k, M):
    torch, q4, dev = env
    rng = np.random.default_rng(T + k + M)
    R = T * k
    for y_bf16 in (True, False):
        Y = rng.standard_normal((R, M)).astype(np.float32)
        Y = ref.bf16(Y) if y_bf16 else Y
        w = rng.uniform(0, 1, (T, k)).astype(np.float32)
        pos = rng.permutation(R).astype(np.int32).reshape(T, k)
        skip = rng.random((T, k)) < 0.1
        pos[skip] = rng.choice([-1, R, 2 ** 30], skip.sum())
        w[skip] = np.nan
        Yd = _dev(env, Y).to(torch.bfloat16 if y_bf16 else torch.float32)
        live = (pos >= 0) & (pos < R)
        term = np.where(live, w, 0).astype(np.float64)[:, :, None] * Y.astype(np.float64)[np.where(live, pos, 0)]
        want = term.sum(1)
        bound = (k + 1) * 2.0 ** -24 * np.abs(term).sum(1)
        for out_bf16 in (True, False):
            out = q4.q4_moe_combine(Yd, _dev(env, w), _dev(env, pos),
                                    out_dtype=torch.bfloat16 if out_bf16 else torch.float32)
            _within(out, want, ref.rounded(want, bound, out_bf16), f"combine {T} {k} {M}")


# ---------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [1, 5, 97])
def test_layer(env, T):
    """Router, gate/up, down and sum in a row, as a model runs them, against
    the 64-bit layer; the rounding of H and Y to bf16 is part of the bound."""
    torch, q4, dev = env
    rng = np.random.default_rng(T)
    E, k, K, F = 6, 2, 192, 128
    M = K
    X = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    logits = rng.standard_normal((T, E)).astype(np.float32)
    g, u, d = _packed(rng, E, F, K), _packed(rng, E, F, K), _packed(rng, E, M, F)
    t = lambda a: _dev(env, a)  # noqa: E731
    ex, w, off, rows, pos = q4.q4_route_topk(t(logits), k)
    H = q4.q4_gemm_grouped(t(g[0]), t(g[1]), t(X).to(torch.bfloat16), off, rows=rows, up=(t(u[0]), t(u[1])))
    Y = q4.q4_gemm_grouped(t(d[0]), t(d[1]), H, off)
    out = q4.q4_moe_combine(Y, w, pos)
    experts, weights, *_ = ref.route(logits, k, "topk")
    lv = q4.codebook()
    want, bound = np.zeros((T, M)), np.zeros((T, M))
    for n in range(T):
        for j in range(k):
            e = experts[n, j]
            Wg, Wu, Wd = (ref.dequantise(lv, m[0][e], m[1][e]) for m in (g, u, d))
            x = X[n:n + 1].astype(np.float64)
            yg, bg = ref.product(Wg, g[1][e], x)
            yu, bu = ref.product(Wu, u[1][e], x)
            h, bh = ref.swiglu(yg, bg, yu, bu)
            bh = ref.rounded(h, bh, True)
            y, by = ref.product(Wd, d[1][e], h)
            by = by + (1 + 2.0 ** -9) * bh @ np.abs(Wd).T
            by = ref.rounded(y, by, True)
            want[n] += weights[n, j] * y[0]
            bound[n] += weights[n, j] * by[0] + 2.0 ** -20 * weights[n, j] * np.abs(y[0])
    _within(out, want, ref.rounded(want, bound, True), f"layer T={T}")
