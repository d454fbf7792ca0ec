"""Low-rank adapters beside a packed projection on the GPU (q4_lora.h), forward
and backward, against plain 64-bit forms and against differences.  The bounds
are those of tests/ragged_reference.py."""
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


class Case:
    def __init__(self, env, M, K, N, r, L, seed, ids="runs", spread=False):
        torch, q4, dev = env
        rng = np.random.default_rng(seed)
        self.codes = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
        s = rng.uniform(0.02, 0.08, (M, K // 64))
        if spread:
            s = s * 2.0 ** rng.integers(-20, 6, (M, 1))
            s[::5] = 0
        self.scales = s.astype(np.float16)
        self.X = ref.bf16(rng.standard_normal((N, K)).astype(np.float32) * rng.choice([0.05, 1.0], (N, 1)))
        self.A = ref.bf16(rng.standard_normal((L, r, K)).astype(np.float32) * K ** -0.5)
        self.B = ref.bf16(rng.standard_normal((L, M, r)).astype(np.float32) * 0.1)
        self.scaling = rng.uniform(0.25, 2, L).astype(np.float32)
        self.dY = ref.bf16(rng.standard_normal((N, M)).astype(np.float32) * 1e-4)
        if ids == "runs":
            i = np.sort(rng.integers(-1, L, N)) if N else np.zeros(0, int)
            i = rng.permutation(L + 1)[i + 1] - 1 if N else i
        elif ids == "none":
            i = np.full(N, -1)
        else:
            i = rng.choice([-1, L, 2 ** 31 - 1, -2 ** 31] + list(range(L)) * 4, N)
        self.ids = np.asarray(i).astype(np.int32)
        bf = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16)  # noqa: E731
        d = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        self.args = (d(self.codes), d(self.scales), bf(self.X), bf(self.A), bf(self.B), d(self.scaling), d(self.ids))
        self.dYd = bf(self.dY)
        f = np.float64
        self.host = (self.X.astype(f), self.A.astype(f), self.B.astype(f), self.scaling.astype(f), self.ids)


def _within(got, want, bound, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    bad = np.abs(got - want) / np.maximum(bound, 1e-300)
    print(f"{what}: worst |err|/bound = {bad.max() if bad.size else 0:.3g}", flush=True)
    assert np.all(np.abs(got - want) <= bound), f"{what}: worst {bad.max()}"


SHAPES = [
    # M, K, N, r, L
    (1, 64, 1, 8, 1),
    (33, 128, 1, 16, 3),
    (70, 256, 7, 8, 4),
    (64, 2048, 32, 16, 9),
    (40, 2112, 3, 24, 2),      # two ranges of K
    (257, 192, 64, 32, 5),
    (130, 320, 65, 40, 3),
    (96, 448, 161, 64, 4),
    (300, 128, 300, 128, 2),
    (523, 192, 513, 16, 6),
    (2048, 128, 100, 8, 1),
    (50, 2112, 2, 16, 2),
    (64, 2048, 1000, 128, 2),  # many chunks, the largest rank
    (130, 320, 1300, 40, 3),   # tile kernel, the shared first product
    (1030, 128, 8300, 72, 3),  # 256 rows a piece
    (300, 1088, 1100, 24, 2),  # runs of K
]


@pytest.mark.parametrize("M,K,N,r,L", SHAPES)
@pytest.mark.parametrize("ids", ["runs", "random", "none"])
def test_forward(env, M, K, N, r, L, ids):
    torch, q4, dev = env
    c = Case(env, M, K, N, r, L, seed=M + K + N + r, ids=ids)
    want, e = ref.lora(q4.codebook(), c.codes, c.scales, *c.host)
    for bf in (True, False):
        y = q4.q4_gemm_lora(*c.args, out_dtype=torch.bfloat16 if bf else torch.float32)
        _within(y, want, ref.rounded(want, e, bf), f"lora {M} {K} {N} {r} {L} {ids}")


@pytest.mark.parametrize("M,K,N,r,L", SHAPES)
@pytest.mark.parametrize("ids", ["runs", "random", "none"])
def test_backward(env, M, K, N, r, L, ids):
    torch, q4, dev = env
    c = Case(env, M, K, N, r, L, seed=M + K + N + r + 1, ids=ids)
    (x, ex), (a, ea), (b, eb) = ref.lora_backward(q4.codebook(), c.codes, c.scales, *c.host, c.dY.astype(np.float64))
    dX, dA, dB = q4.q4_gemm_lora_backward(c.dYd, *c.args)
    what = f"{M} {K} {N} {r} {L} {ids}"
    _within(dX, x, ref.rounded(x, ex, True), "dX " + what)
    _within(dA, a, ea + 2.0 ** -24 * np.abs(a) + 1e-37, "dA " + what)
    _within(dB, b, eb + 2.0 ** -24 * np.abs(b) + 1e-37, "dB " + what)
    again = q4.q4_gemm_lora_backward(c.dYd, *c.args)
    for p, q in zip((dX, dA, dB), again):
        assert torch.equal(p, q)
    one = q4.q4_gemm_lora_backward(c.dYd, *c.args, need_adapters=False)
    two = q4.q4_gemm_lora_backward(c.dYd, *c.args, need_dX=False)
    assert torch.equal(one[0], dX) and one[1] is None and two[0] is None
    assert torch.equal(two[1], dA) and torch.equal(two[2], dB)


@pytest.mark.parametrize("N", [5, 200, 1100])
def test_scales_of_every_magnitude(env, N):
    torch, q4, dev = env
    c = Case(env, 90, 256, N, 8, 2, seed=4, spread=True)
    want, e = ref.lora(q4.codebook(), c.codes, c.scales, *c.host)
    _within(q4.q4_gemm_lora(*c.args, out_dtype=torch.float32), want, ref.rounded(want, e, False), "forward")
    (x, ex), _, _ = ref.lora_backward(q4.codebook(), c.codes, c.scales, *c.host, c.dY.astype(np.float64))
    _within(q4.q4_gemm_lora_backward(c.dYd, *c.args)[0], x, ref.rounded(x, ex, True), "dX")


def test_gradients_against_differences(env):
    """The loss sum(dY * Y) moves by the gradient times a step: Y from the
    64-bit form, whose central difference over a linear argument is exact."""
    torch, q4, dev = env
    c = Case(env, 48, 128, 6, 8, 2, seed=21, ids="runs")
    dX, dA, dB = (g.float().cpu().numpy().astype(np.float64) for g in q4.q4_gemm_lora_backward(c.dYd, *c.args))
    dY = c.dY.astype(np.float64)
    X, A, B, s, ids = c.host
    loss = lambda X, A, B: float((dY * ref.lora(q4.codebook(), c.codes, c.scales, X, A, B, s, ids)[0]).sum())  # noqa: E731
    rng = np.random.default_rng(1)
    for k, (g, tol) in enumerate(((dX, 2.0 ** -7), (dA, 1e-5), (dB, 1e-5))):
        v = rng.standard_normal(g.shape)
        at = [X, A, B]
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + 0.5 * v, at[k] - 0.5 * v
        diff = loss(*up) - loss(*down)
        assert abs(diff - (g * v).sum()) <= tol * np.abs(g * v).sum()


def test_no_adapters_and_no_tokens(env):
    torch, q4, dev = env
    c = Case(env, 40, 128, 9, 8, 2, seed=2)
    e = torch.empty
    none = (e((0, 8, 128), dtype=torch.bfloat16, device=dev), e((0, 40, 8), dtype=torch.bfloat16, device=dev),
            e(0, device=dev), c.args[6])
    y = q4.q4_gemm_lora(*c.args[:3], *none)
    off = q4.q4_gemm_lora(*c.args[:6], torch.full_like(c.args[6], -1))
    assert torch.equal(y, off)
    dX, dA, dB = q4.q4_gemm_lora_backward(c.dYd, *c.args[:3], *none)
    ref_dX = q4.q4_gemm_lora_backward(c.dYd, *c.args[:6], torch.full_like(c.args[6], -1))
    assert torch.equal(dX, ref_dX[0]) and dA.numel() == 0
    assert not ref_dX[1].any() and not ref_dX[2].any()
    zero = tuple(a[:0] if i in (2, 6) else a for i, a in enumerate(c.args))
    assert q4.q4_gemm_lora(*zero).shape == (0, 40)
    dX, dA, dB = q4.q4_gemm_lora_backward(c.dYd[:0], *zero)
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


@pytest.mark.parametrize("N", [4, 150, 1100])
def test_one_token_that_is_not_finite(env, N):
    torch, q4, dev = env
    c = Case(env, 64, 256, N, 16, 2, seed=9, ids="random")
    y0 = q4.q4_gemm_lora(*c.args, out_dtype=torch.float32)
    g0 = q4.q4_gemm_lora_backward(c.dYd, *c.args)[0]
    x = c.args[2].clone()
    x[2, 7] = float("inf")
    y1 = q4.q4_gemm_lora(*c.args[:2], x, *c.args[3:], out_dtype=torch.float32)
    dy = c.dYd.clone()
    dy[2, 7] = float("nan")
    g1 = q4.q4_gemm_lora_backward(dy, *c.args)[0]
    keep = torch.arange(N, device=dev) != 2
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(g0[keep], g1[keep])
    assert not torch.isfinite(y1[2]).all() and not torch.isfinite(g1[2].float()).any()


@pytest.mark.parametrize("M,K,N", [(200, 2112, 6), (300, 256, 150), (300, 256, 1100)])
def test_captured_with_other_work_between(env, M, K, N):
    torch, q4, dev = env
    c = Case(env, M, K, N, 16, 3, seed=N)
    y0 = q4.q4_gemm_lora(*c.args)
    g0 = q4.q4_gemm_lora_backward(c.dYd, *c.args)
    side = torch.cuda.Stream()
    y = torch.empty_like(y0)
    g = [torch.empty_like(t) for t in g0]
    ws = torch.empty(q4.q4_gemm_lora_ws_bytes(M, K, N, 16, 3), dtype=torch.uint8, device=dev)
    wb = torch.empty(q4.q4_gemm_lora_backward_ws_bytes(M, K, N, 16, 3), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        q4.q4_gemm_lora(*c.args, Y=y, workspace=ws, stream=side)
        q4.q4_gemm_lora_backward(c.dYd, *c.args, dX=g[0], dA=g[1], dB=g[2], workspace=wb, stream=side)
    for rep in range(3):
        y.fill_(float("nan"))
        for t in g:
            t.fill_(float("nan"))
        wb.fill_(255)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0), rep
        for p, q in zip(g, g0):
            assert torch.equal(p, q), rep
        q4.q4_gemm_lora(*c.args)
