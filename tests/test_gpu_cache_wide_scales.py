"""Attention over caches whose scales differ by many powers of two: between the
blocks of a row, between keys, and between keys that a row sees and keys that
others of its tile see.  Each output is as near as its own scales allow: keys
that a row does not see, blocks other than its own and keys of negligible
weight do not cost it bits.  Bounds: tests/cache_reference.py, whose roundings
are all relative to the seen values."""
import numpy as np
import pytest

from test_gpu_cache import Batch, _rows_of, env, to_cache, within  # noqa: F401
import cache_reference as ref

pytestmark = pytest.mark.gpu


def logarithmic(rng, lo, hi, shape):
    return np.exp(rng.uniform(np.log(lo), np.log(hi), shape)).astype(np.float16)


def batch(env, lens, new, heads, G, D, seed, low=0.001, high=0.5, key_low=0.001, key_high=0.02, slack=1):
    b = Batch(env, lens, new, heads, G, D, 16, seed, slack=slack)
    rng = np.random.default_rng(seed)
    b.planes["v_scales"] = logarithmic(rng, low, high, b.planes["v_scales"].shape)
    b.planes["k_scales"] = logarithmic(rng, key_low, key_high, b.planes["k_scales"].shape)
    return b


def renew(env, b):
    b.dev = (b.dev[0], to_cache(env, b.planes)) + b.dev[2:]
    return b


SHAPES = [  # lens, new tokens, heads, G, D
    ([170, 99], [80, 40], 2, 4, 128),
    ([260], [200], 1, 2, 64),
    ([150, 60], [60, 40], 1, 1, 256),
    ([400, 130], [120, 50], 1, 2, 192),
    ([1200], [50], 1, 1, 256),               # keys dealt to several workgroups
    ([2600, 700], [150, 300], 1, 2, 128),
    ([170, 99], [80, 1], 2, 4, 128),
    ([170, 99], [5, 1], 2, 4, 128),          # drafts: rows of a tile of keys see different ones
    ([700, 90], [7, 5], 1, 2, 192),
    ([2100, 40], [4, 3], 1, 3, 64),
    ([700, 90], [9, 3], 1, 7, 128),
    ([600, 1500], [8, 2], 1, 4, 256),
    ([400, 300], [30, 2], 1, 2, 64),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("where", ["causal", "window"])
def test_large_keys_that_a_row_does_not_see(env, i, side, where):
    """A key of scale 65504 among the new tokens, behind half of them, or in the
    window of the first rows and before that of the later ones."""
    torch, q4, dev = env
    lens, new, heads, G, D = SHAPES[i]
    b = batch(env, lens, new, heads, G, D, 600 + i, slack=80 if lens[0] > 1024 else 1)
    window = 40 if where == "window" else 0
    bad = lens[0] - max(1, new[0] // 2)
    if window:
        bad = lens[0] - new[0] + max(1, new[0] // 2) - window   # the later half's windows begin behind it
    assert 0 <= bad < lens[0]
    ids, at = _rows_of(b, 0, [bad])
    b.planes[side + "_scales"][ids[0], :, at[0]] = 65504
    renew(env, b)
    out, lse = b.check(env, f"{side} {where}", window=window, dtype="float32")
    # The rows that do not see it, against a cache without it.
    pos = lens[0] - new[0] + np.arange(new[0])
    blind = np.ones(b.q.shape[0], bool)
    blind[:new[0]] = (pos < bad) | ((window > 0) & (pos - window + 1 > bad))
    assert blind[:new[0]].any() and not blind[:new[0]].all()
    b.planes[side + "_scales"][ids[0], :, at[0]] = 0.01
    renew(env, b)
    clean, clean_lse = b.check(env, "without", window=window, dtype="float32")
    o, bound, l, lb, _ = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, b.offsets, True, window, None, False)
    for got in (out, clean):
        within(got[torch.from_numpy(blind).to(dev)], o[blind], bound[blind], "rows that do not see it")
    within(lse[torch.from_numpy(blind).to(dev)], l[blind], lb[blind], "their lse")


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("low,high", [(2.0 ** -24, 2.0 ** -20), (2.0 ** -24, 2.0 ** 12), (2.0 ** -12, 2.0 ** 12)])
def test_scales_of_every_size_side_by_side(env, i, low, high):
    lens, new, heads, G, D = SHAPES[i]
    b = renew(env, batch(env, lens, new, heads, G, D, 700 + i, low, high, key_low=2.0 ** -24, key_high=0.25, slack=80))
    b.check(env, f"scales {low} to {high}", dtype="float32")
    b.check(env, f"scales {low} to {high}", dtype="float32", window=33)


@pytest.mark.parametrize("lens,new,heads,G,D", SHAPES + [
    ([300, 200, 90], [1, 1, 1], 2, 8, 128), ([4000, 9], [1, 1], 1, 5, 256), ([5000, 100], [1, 1], 2, 2, 128)])
def test_blocks_of_a_row_far_apart(env, lens, new, heads, G, D):
    """The first block's values 2^16 to 2^30 times the last one's: every block's
    outputs within its own bound, in keys alike and in one key of 37."""
    rng = np.random.default_rng(5)
    for large, small, every in ((60000.0, 2.0 ** -14, 1), (4.0, 2.0 ** -20, 1), (65504.0, 0.0015, 37), (2.0 ** 10, 2.0 ** -10, 64)):
        b = batch(env, lens, new, heads, G, D, 800 + D, small, 1.9 * small, slack=80)
        v = b.planes["v_scales"]
        for s in range(len(lens)):
            ids, at = _rows_of(b, s, np.arange(0, lens[s], every))
            v[ids, :, at, 0] = np.float16(large) * rng.uniform(0.5, 1.0, (len(ids), heads)).astype(np.float16)
        renew(env, b)
        b.check(env, f"blocks {large} {small} every {every}", dtype="float32")


@pytest.mark.parametrize("lens,new,heads,G,D", [([900, 300], [90, 80], 1, 2, 128), ([700], [300], 2, 2, 64),
                                                ([1100], [40], 1, 2, 256), ([1500, 40], [6, 2], 2, 2, 64),
                                                ([1100], [1], 1, 4, 128), ([1100], [9], 1, 7, 128)])
def test_stretches_of_large_and_small_values(env, lens, new, heads, G, D):
    """Tiles of large values, of small ones and of both in turn: what has been
    summed is carried from one power of two to the next, up and down."""
    torch, q4, dev = env
    b = batch(env, lens, new, heads, G, D, 900 + D, slack=80)
    rng = np.random.default_rng(9)
    for s in range(len(lens)):
        for first, size in ((0, 0.01), (130, 30000.0), (200, 0.01), (270, 2.0 ** -20), (400, 0.01), (470, 3000.0), (500, 0.01)):
            keys = np.arange(first, min(first + (130 if first != 200 else 70), lens[s]))
            if len(keys):
                ids, at = _rows_of(b, s, keys)
                b.planes["v_scales"][ids, :, at] = (size * rng.uniform(0.5, 1, (len(keys), heads, D // 64))).astype(np.float16)
    renew(env, b)
    b.check(env, "stretches", dtype="float32")
    b.check(env, "stretches", dtype="float32", causal=False)


@pytest.mark.parametrize("new", [[80, 50], [80, 1], [4, 1], [1, 1]])
def test_large_values_of_no_weight(env, new):
    """A seen key of the largest value scale whose weight is far below what its
    output would notice, and outputs from small values beside it."""
    b = batch(env, [170, 99], new, 1, 2, 128, 31, 0.001, 0.003, key_low=0.01, key_high=0.02)
    ids, at = _rows_of(b, 0, [20])
    row = (ids[0], 0, at[0])
    # A key opposite to every query: their first dimension is large and positive.
    b.q[:, :, 0] = 200.0
    b.planes["k_codes"][row] = 0x88
    b.planes["k_codes"][row + (0,)] = 0x80
    b.planes["k_zeros"][row] = 8
    b.planes["k_scales"][row] = 1.0      # its score: -8 * 200 / sqrt(128) below the others'
    b.planes["v_scales"][row] = 65504
    torch, q4, dev = env
    b.dev = (torch.from_numpy(b.q).to(dev).to(torch.bfloat16),) + b.dev[1:]
    renew(env, b)
    out, _ = b.check(env, "no weight", dtype="float32")
    assert out[:new[0]].abs().max() < 0.1


@pytest.mark.parametrize("lens,new,heads,G,D", SHAPES)
def test_not_finite_among_scales_far_apart(env, lens, new, heads, G, D):
    """A NaN scale of one block of one value in a tile of scales far apart: its
    block is NaN in the rows that see it, all else within the bound."""
    b = batch(env, lens, new, heads, G, D, 950 + D, 2.0 ** -20, 2.0 ** 6, slack=80)
    bad = lens[0] - max(1, new[0] // 2)
    ids, at = _rows_of(b, 0, [bad])
    scale = b.planes["v_scales"][ids[0], :, at[0], -1].copy()
    b.planes["v_scales"][ids[0], :, at[0], -1] = np.nan
    renew(env, b)
    torch, q4, dev = env
    o2 = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, out_dtype=torch.float32)
    o1, _ = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, out_dtype=torch.float32, return_lse=True)
    b.planes["v_scales"][ids[0], :, at[0], -1] = scale
    want, bound, _, _, _ = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, b.offsets, out_bf16=False)
    sees = np.zeros(b.q.shape[0], bool)
    sees[:new[0]] = lens[0] - new[0] + np.arange(new[0]) >= bad
    for got in (o1, o2):
        g = got.cpu().numpy()
        assert np.isnan(g[sees][..., D - 64:]).all() and np.isfinite(g[~sees]).all()
        within(got[torch.from_numpy(~sees).to(dev)], want[~sees], bound[~sees], "rows that do not see it")
        if D > 64:
            within(got[torch.from_numpy(sees).to(dev)][..., :D - 64], want[sees][..., :D - 64], bound[sees][..., :D - 64], "its other blocks")


@pytest.mark.parametrize("lens,new,heads,G,D", [([900, 300], [90, 80], 1, 2, 128), ([300, 170], [1, 1], 2, 4, 128), ([2100, 40], [4, 3], 1, 3, 64),
                                                ([400], [60], 1, 1, 256)])
def test_captured_calls_as_the_scales_grow_apart(env, lens, new, heads, G, D):
    """One captured call, replayed as the cache's scales change in place: close
    together, one far from the others, far apart everywhere, all zero."""
    torch, q4, dev = env
    b = renew(env, batch(env, lens, new, heads, G, D, 970 + D, 0.1, 0.5, slack=80))
    rng = np.random.default_rng(4)
    out = torch.empty(b.q.shape, dtype=torch.float32, device=dev)
    lse = torch.empty(b.q.shape[:2], device=dev)
    need = q4.q4_cache_attend_ws_bytes(b.q.shape[0], heads * G, heads, D, len(lens), b.max_q)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    kw = dict(q_offsets=b.offsets_dev, max_q=b.max_q)

    def both(o, l):
        q4.q4_cache_attend(*b.dev, out=o, workspace=ws, **kw)
        q4.q4_cache_attend(*b.dev, out=torch.empty_like(o), lse=l, workspace=ws, **kw)

    both(out, lse)
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            both(out, lse)
    torch.cuda.synchronize()
    shape = b.planes["v_scales"].shape
    steps = [logarithmic(rng, 0.1, 0.5, shape) for _ in range(4)]
    ids, at = _rows_of(b, 0, [37])
    steps[1][ids[0], :, at[0]] = 65504
    steps[2] = logarithmic(rng, 2.0 ** -24, 2.0 ** 10, shape)
    steps[3][:] = 0
    for n, scales in enumerate(steps + steps[:1]):
        b.planes["v_scales"] = scales
        b.cache = b.dev[1]
        b.cache.v_scales.copy_(torch.from_numpy(scales))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager, eager_lse = torch.empty_like(out), torch.empty_like(lse)
        both(eager, eager_lse)
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse), n
        want, bound, l, lb, _ = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, b.offsets, out_bf16=False)
        within(out, want, bound, f"replay {n}")
        within(lse, l, lb, f"replay {n} lse")


@pytest.mark.parametrize("lens,new,heads,G,D", SHAPES)
def test_hidden_pages_among_scales_far_apart(env, lens, new, heads, G, D):
    torch, q4, dev = env
    b = batch(env, lens, new, heads, G, D, 990 + D, 2.0 ** -20, 2.0 ** 10, slack=80)
    for row in b.table:
        row[1:6:2] = (-1, len(b.planes["k_codes"]), 2 ** 31 - 1)
    renew(env, b)
    b.dev = b.dev[:2] + (torch.from_numpy(b.table).to(dev), b.dev[3])
    b.check(env, "hidden", dtype="float32")
    b.check(env, "hidden", dtype="float32", window=50)
