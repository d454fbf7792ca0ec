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
