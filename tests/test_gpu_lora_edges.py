"""Calls of the adapters' entry points at the borders of their contract
(q4_lora.h), on the GPU, against plain 64-bit forms.  The bounds are those of
tests/ragged_reference.py."""
import numpy as np
import pytest

import ragged_reference as ref
from test_gpu_experts_edges import _same_kind
from test_gpu_lora import Case, _within, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _plain(levels, c, X, A, B, s, dY=None):
    """The formulas in 64 bits, product by product, so that an infinity times a
    zero is NaN only where the formula has that product."""
    W = ref.dequantise(levels, c.codes, c.scales)
    with np.errstate(invalid="ignore", over="ignore"):
        Y = X @ W.T
        dA, dB = np.zeros(A.shape), np.zeros(B.shape)
        dX = dY @ W
        for n, a in enumerate(c.ids):
            if not 0 <= a < len(A):
                continue
            t, u = s[a] * (A[a] @ X[n]), s[a] * (B[a].T @ dY[n])
            Y[n] += B[a] @ t
            dX[n] += u @ A[a]
            dA[a] += np.outer(u, X[n])
            dB[a] += np.outer(dY[n], t)
    return Y, dX, dA, dB


# M, K, N, r: the row, chunk and tile kernels, tiles in runs of K, dX with and
# without planes, ranks of one and of several matrix-core steps.
MIXED = [(40, 192, 2, 8), (64, 256, 4, 16), (64, 256, 30, 8), (300, 256, 150, 24), (40, 256, 300, 16), (300, 256, 1100, 16),
         (64, 192, 1100, 8), (300, 1088, 1100, 40), (2048, 128, 1030, 16), (1030, 128, 8300, 24)]


def _spoiled(env, M, K, N, r, where):  # noqa: F811
    """A case of four adapters, and the same call with an infinity or a NaN in
    two of them: (case, arguments, (A, B, scaling), tokens of the others)."""
    torch, q4, dev = env
    c = Case(env, M, K, N, r, 4, seed=M + N + r, ids="random")
    if N == 2:
        c.ids = np.array([1, 2], np.int32)
        c.args = c.args[:6] + (torch.from_numpy(c.ids).to(dev),)
    A, B, s = (a.copy() for a in (c.A, c.B, c.scaling))
    if where == "A":
        A[1, 2, 5], A[2, r - 1, K - 1] = np.inf, -np.inf
    elif where == "B":
        B[1, 7, 3], B[2, M - 1, r - 1], B[2, 3, 0] = np.inf, -np.inf, np.nan
    else:
        s[1], s[2] = np.inf, np.nan
    bf = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16)  # noqa: E731
    args = c.args[:3] + (bf(A), bf(B), torch.from_numpy(s).to(dev), c.args[6])
    keep = torch.from_numpy((c.ids != 1) & (c.ids != 2)).to(dev)
    return c, args, (A, B, s), keep


@pytest.mark.parametrize("M,K,N,r", MIXED)
@pytest.mark.parametrize("where", ["A", "B", "scaling"])
def test_an_adapter_that_is_not_finite_leaves_other_tokens(env, M, K, N, r, where):  # noqa: F811
    """An infinity or a NaN in one adapter: tokens of other adapters, and of
    none, keep their bits."""
    torch, q4, dev = env
    c, args, _, keep = _spoiled(env, M, K, N, r, where)
    y0 = q4.q4_gemm_lora(*c.args, out_dtype=torch.float32)
    y1 = q4.q4_gemm_lora(*args, out_dtype=torch.float32)
    assert torch.equal(y0[keep], y1[keep])
    assert not torch.isfinite(y1[~keep]).all()


@pytest.mark.parametrize("M,K,N,r", MIXED)
@pytest.mark.parametrize("where", ["A", "B", "scaling"])
def test_an_adapter_that_is_not_finite_leaves_other_gradients(env, M, K, N, r, where):  # noqa: F811
    torch, q4, dev = env
    c, args, _, keep = _spoiled(env, M, K, N, r, where)
    g0 = q4.q4_gemm_lora_backward(c.dYd, *c.args)
    g1 = q4.q4_gemm_lora_backward(c.dYd, *args)
    assert torch.equal(g0[0][keep], g1[0][keep])
    for a in (0, 3):
        assert torch.equal(g0[1][a], g1[1][a]) and torch.equal(g0[2][a], g1[2][a])


@pytest.mark.parametrize("M,K,N,r", MIXED)
@pytest.mark.parametrize("where", ["A", "B", "scaling"])
def test_an_adapter_that_is_not_finite_gives_what_the_formula_gives(env, M, K, N, r, where):  # noqa: F811
    """Infinities of the right sign, and NaN only where the formula has one."""
    torch, q4, dev = env
    c, args, (A, B, s), _ = _spoiled(env, M, K, N, r, where)
    y = q4.q4_gemm_lora(*args, out_dtype=torch.float32)
    g = q4.q4_gemm_lora_backward(c.dYd, *args)
    f = np.float64
    want = _plain(q4.codebook(), c, c.X.astype(f), A.astype(f), B.astype(f), s.astype(f), c.dY.astype(f))
    for got, w, what in zip((y,) + tuple(g), want, ("Y", "dX", "dA", "dB")):
        _same_kind(got, w, what)


@pytest.mark.parametrize("M,K,N,r", MIXED)
def test_scaling_of_zero_and_below(env, M, K, N, r):  # noqa: F811
    """s B x = |s| (sign(s) B) x, so that the reference's bounds keep their sign."""
    torch, q4, dev = env
    c = Case(env, M, K, N, r, 3, seed=M + N, ids="random")
    s = np.array([-0.75, 0.0, 1.5], np.float32)
    args = c.args[:5] + (torch.from_numpy(s).to(dev), c.args[6])
    X, A, B, _, ids = c.host
    sign = np.sign(s.astype(np.float64))[:, None, None]
    host = (X, A, B * np.where(sign == 0, 1, sign), np.abs(s.astype(np.float64)), ids)
    want, e = ref.lora(q4.codebook(), c.codes, c.scales, *host)
    _within(q4.q4_gemm_lora(*args, out_dtype=torch.float32), want, ref.rounded(want, e, False), "forward")
    (x, ex), (a, ea), (b, eb) = ref.lora_backward(q4.codebook(), c.codes, c.scales, *host, c.dY.astype(np.float64))
    dX, dA, dB = q4.q4_gemm_lora_backward(c.dYd, *args)
    _within(dX, x, ref.rounded(x, ex, True), "dX")
    _within(dA, a, ea + 2.0 ** -24 * np.abs(a) + 1e-37, "dA")
    b, eb = b * np.where(sign == 0, 1, sign), eb
    _within(dB, b, eb + 2.0 ** -24 * np.abs(b) + 1e-37, "dB")


@pytest.mark.parametrize("M,K,N", [(66, 192, 5), (66, 192, 300), (300, 256, 1100), (1030, 64, 70)])
@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 60, 3e38])
def test_gradients_beside_a_packed_row_of_zeros(env, M, K, N, big):  # noqa: F811
    """A packed row whose scales are all 0 adds nothing to dX, however large
    its dY is."""
    torch, q4, dev = env
    c = Case(env, M, K, N, 8, 2, seed=N + M, ids="random")
    c.scales[3] = 0
    c.B[:, 3] = 0                       # (u has no part of it either)
    c.dY[:, 3] = ref.bf16(np.float32(big))
    bf = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16)  # noqa: E731
    args = (c.args[0], torch.from_numpy(c.scales).to(dev), c.args[2], c.args[3], bf(c.B), c.args[5], c.args[6])
    host = (c.host[0], c.host[1], c.B.astype(np.float64), c.host[3], c.host[4])
    (x, ex), _, _ = ref.lora_backward(q4.codebook(), c.codes, c.scales, *host, c.dY.astype(np.float64))
    dX, _, _ = q4.q4_gemm_lora_backward(bf(c.dY), *args, need_adapters=False)
    _within(dX, x, ref.rounded(x, ex, True), f"dX beside a row of zeros, {big}")


@pytest.mark.parametrize("M,K,N,r", MIXED)
def test_one_infinite_token(env, M, K, N, r):  # noqa: F811
    """An infinity in a token's row, also in its last values, where a kernel's
    steps reach past the row."""
    torch, q4, dev = env
    c = Case(env, M, K, N, r, 3, seed=M + r, ids="random")
    X, dY = c.X.copy(), c.dY.copy()
    X[0, K - 1], X[N - 1, K - 33] = np.inf, -np.inf
    dY[0, M - 1], dY[N - 1, 3] = np.inf, -np.inf
    bf = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16)  # noqa: E731
    y = q4.q4_gemm_lora(*c.args[:2], bf(X), *c.args[3:], out_dtype=torch.float32)
    g = q4.q4_gemm_lora_backward(bf(dY), *c.args[:2], bf(X), *c.args[3:])
    f = np.float64
    want = _plain(q4.codebook(), c, X.astype(f), c.A.astype(f), c.B.astype(f), c.scaling.astype(f), dY.astype(f))
    for got, w, what in zip((y,) + tuple(g), want, ("Y", "dX", "dA", "dB")):
        _same_kind(got, w, what)


@pytest.mark.parametrize("M,K,N", [(66, 192, 5), (72, 192, 300), (300, 256, 1100), (1030, 64, 70), (14000, 64, 3)])
@pytest.mark.parametrize("small", [(0, 1), (2, 3, 4, 5, 6, 7), (0, 2, 4, 6), (5,)])
def test_gradients_of_rows_of_unlike_scales(env, M, K, N, small):  # noqa: F811
    """Among eight neighbouring packed rows some have scales 2^-12 of the
    others': each row counts with its own power of two."""
    torch, q4, dev = env
    c = Case(env, M, K, N, 8, 2, seed=N + M, ids="random")
    c.scales[np.isin(np.arange(M) % 8, small)] *= np.float16(2.0 ** -12)
    args = (c.args[0], torch.from_numpy(c.scales).to(dev)) + c.args[2:]
    (x, ex), _, _ = ref.lora_backward(q4.codebook(), c.codes, c.scales, *c.host, c.dY.astype(np.float64))
    dX, _, _ = q4.q4_gemm_lora_backward(c.dYd, *args, need_adapters=False)
    _within(dX, x, ref.rounded(x, ex, True), f"dX of rows of unlike scales, {small}")


# M, K, N, r, L: the longest rows, many packed rows, many adapters, the largest rank.
LARGEST = [(5, 131072, 1, 8, 2), (5, 131072, 20, 16, 2), (3, 131008, 300, 8, 1), (70000, 64, 3, 8, 2), (30, 64, 3000, 8, 1024),
           (40, 192, 700, 16, 700), (70, 192, 1500, 128, 2), (130, 64, 70, 128, 40)]


@pytest.mark.parametrize("M,K,N,r,L", LARGEST)
def test_largest(env, M, K, N, r, L):  # noqa: F811
    torch, q4, dev = env
    c = Case(env, M, K, N, r, L, seed=M + K + N + r, ids="random")
    want, e = ref.lora(q4.codebook(), c.codes, c.scales, *c.host)
    _within(q4.q4_gemm_lora(*c.args, out_dtype=torch.float32), want, ref.rounded(want, e, False), "forward")
    (x, ex), (a, ea), (b, eb) = ref.lora_backward(q4.codebook(), c.codes, c.scales, *c.host, c.dY.astype(np.float64))
    dX, dA, dB = q4.q4_gemm_lora_backward(c.dYd, *c.args)
    _within(dX, x, ref.rounded(x, ex, True), "dX")
    _within(dA, a, ea + 2.0 ** -24 * np.abs(a) + 1e-37, "dA")
    _within(dB, b, eb + 2.0 ** -24 * np.abs(b) + 1e-37, "dB")


@pytest.mark.parametrize("M,K,N,r", [(64, 256, 4, 16), (200, 2112, 30, 24), (300, 1088, 1100, 40)])
def test_two_calls_at_once(env, M, K, N, r):  # noqa: F811
    """Calls on two streams without a wait between them, each with scratch of
    its own: the bits of calls by themselves."""
    torch, q4, dev = env
    cases = [Case(env, M, K, N, r, 3, seed=s, ids="random") for s in (1, 2)]
    alone = [(q4.q4_gemm_lora(*c.args),) + q4.q4_gemm_lora_backward(c.dYd, *c.args) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for c, s, g in zip(cases, streams, got):
            g.append((q4.q4_gemm_lora(*c.args, stream=s),) + q4.q4_gemm_lora_backward(c.dYd, *c.args, stream=s))
    torch.cuda.synchronize()
    for g, want in zip(got, alone):
        for out in g:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
