"""The 4-bit key/value cache on the GPU (q4_cache.h): appended rows bit for bit,
rows read back, and attention, against plain 64-bit forms.  The bounds are
those of tests/cache_reference.py."""
import numpy as np
import pytest

import cache_reference as ref

pytestmark = pytest.mark.gpu

PLANES = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales", "v_zeros")


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible: SKIP (not a pass)")
    import bit_weight_gemv_amd as q4
    q4.lib()
    return torch, q4, torch.device("cuda:0")


def to_cache(env, planes):
    torch, q4, dev = env
    return q4.KVCache(*(torch.from_numpy(planes[n]).to(dev) for n in PLANES))


def of_cache(cache):
    return {n: getattr(cache, n).cpu().numpy() for n in PLANES}


def random_planes(rng, pages, heads, page, D, spread=False):
    out = {}
    for x in "kv":
        out[x + "_codes"] = rng.integers(0, 256, (pages, heads, page, D // 2), dtype=np.uint8)
        s = rng.uniform(0.1, 0.5, (pages, heads, page, D // 64))
        if spread:
            s = s * 2.0 ** rng.integers(-8, 3, s.shape)
            s[rng.random(s.shape) < 0.05] = 0
        out[x + "_scales"] = s.astype(np.float16)
        out[x + "_zeros"] = rng.integers(0, 16, s.shape).astype(np.float16)
    return out


def within(got, want, bound, what):
    got = got.float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= bound) | (got == want)
        worst = np.nanmax(np.where(got == want, 0, np.abs(got - want)) / bound) if got.size else 0
    print(f"{what}: worst |err|/bound = {worst:.3g}", flush=True)
    assert ok.all(), f"{what}: worst {worst}"


APPEND = [  # T, heads, q_heads, D, page, rot, interleaved, fp32
    (1, 2, 16, 128, 16, 128, False, True),
    (7, 3, 0, 64, 32, 64, True, False),
    (61, 8, 40, 128, 16, 64, True, False),
    (33, 1, 5, 192, 64, 96, False, True),
    (19, 4, 4, 256, 16, 256, False, False),
    (5, 12, 12, 64, 128, 0, False, True),
    (1100, 2, 4, 128, 64, 128, False, False),
    (40, 2, 2, 192, 16, 16, True, True),
]


@pytest.mark.parametrize("T,heads,qh,D,page,rot,inter,f32", APPEND)
def test_append_is_the_formula_bit_for_bit(env, T, heads, qh, D, page, rot, inter, f32):
    torch, q4, dev = env
    rng = np.random.default_rng(T * 7 + D + rot)
    pages = -(-T * 5 // (4 * page)) + 1
    planes = random_planes(rng, pages, heads, page, D)
    cache = to_cache(env, planes)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    skip = rng.random(T) < 0.15
    given = np.where(skip, rng.choice([-1, pages * page, 2 ** 31 - 1, -2 ** 31], T), slots).astype(np.int32)
    x = rng.standard_normal((T, qh + 2 * heads, D)).astype(np.float32) * rng.choice([1e-3, 1.0, 30.0], (T, 1, 1)).astype(np.float32)
    x[rng.random((T, qh + 2 * heads)) < 0.05] = 0
    if not f32:
        x = ref.bf16(x)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    freq = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    xd = torch.from_numpy(x).to(dev)
    xd = xd if f32 else xd.to(torch.bfloat16)
    q = q4.q4_cache_append(cache, xd[:, qh:qh + heads], xd[:, qh + heads:], torch.from_numpy(given).to(dev),
                           torch.from_numpy(pos).to(dev), torch.from_numpy(freq).to(dev), interleaved=inter, amplitude=1.25,
                           q=xd[:, :qh] if qh else None)
    torch.cuda.synchronize()
    want = {n: p.copy() for n, p in planes.items()}
    for side, new in (("k", ref.rotate(x[:, qh:qh + heads], pos, freq, inter, 1.25)), ("v", x[:, qh + heads:].astype(np.float64))):
        for name, r in zip(("codes", "scales", "zeros"), ref.pack(new)):
            for t in np.flatnonzero(~skip):
                want[f"{side}_{name}"][slots[t] // page, :, slots[t] % page] = r[t]
    got = of_cache(cache)
    for n in PLANES:
        same = got[n] == want[n]
        assert same.all(), (n, int((~same).sum()))
    if qh:
        w = ref.rotate(x[:, :qh], pos, freq, inter, 1.25)
        # Two rounded products and a sum of fp32 factors, then half a bf16 step.
        pairs = np.abs(ref.rotate(np.abs(x[:, :qh]), 0 * pos, freq, inter, 1.0)).astype(np.float64)
        half = rot // 2
        if inter:
            pairs[..., 0:rot:2] = pairs[..., 1:rot:2] = pairs[..., 0:rot:2] + pairs[..., 1:rot:2]
        else:
            pairs[..., :half] = pairs[..., half:rot] = pairs[..., :half] + pairs[..., half:rot]
        pairs[..., rot:] = 0
        e = 2.0 ** -22 * 1.25 * pairs
        within(q, w, 2.0 ** -8 * (np.abs(w) + e) + e + 1e-37, "rotated q")
    else:
        assert q is None


def test_append_blocks_that_are_not_finite(env):
    torch, q4, dev = env
    rng = np.random.default_rng(5)
    cache = to_cache(env, random_planes(rng, 2, 2, 16, 128))
    k = rng.standard_normal((6, 2, 128)).astype(np.float32)
    v = k.copy()
    k[0, 0, 3], k[1, 1, 127], k[2, 0, 64] = np.nan, np.inf, -np.inf
    v[3, 0, 5], v[3, 0, 6] = 3e38, -3e38       # their distance passes fp32
    v[4, 1, 70] = 1e6                           # the scale rounds to an infinity
    v[5, :, :64] = 15 * 65504 * np.float32(0.9999)  # the largest that does not
    v[5, 1, 64:] = 1e-9                         # the scale rounds to zero
    slots = np.arange(6, dtype=np.int32) * 5
    q4.q4_cache_append(cache, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), torch.from_numpy(slots).to(dev))
    got = of_cache(cache)
    for side, x in (("k", k), ("v", v)):
        for name, r in zip(("codes", "scales", "zeros"), ref.pack(x)):
            g = got[f"{side}_{name}"][slots // 16, :, slots % 16]
            assert np.array_equal(g, r, equal_nan=name == "scales"), (side, name)
    kr, vr = q4.q4_cache_read(cache, torch.from_numpy(slots).to(dev), out_dtype=torch.float32)
    kr = kr.cpu().numpy()
    assert np.isnan(kr[0, 0, :64]).all() and np.isfinite(kr[0, 0, 64:]).all() and np.isfinite(kr[0, 1]).all()
    assert (vr[5, 1, 64:] == 0).all()


@pytest.mark.parametrize("n,heads,D,page,dtype", [(1, 1, 64, 16, "bfloat16"), (37, 12, 64, 32, "float32"),
                                                  (100, 8, 128, 64, "bfloat16"), (9, 3, 192, 16, "float32"),
                                                  (300, 2, 256, 128, "bfloat16"), (4099, 9, 64, 16, "bfloat16"),
                                                  (5000, 8, 192, 32, "float32")])
def test_read_is_the_rows(env, n, heads, D, page, dtype):
    torch, q4, dev = env
    rng = np.random.default_rng(n)
    planes = random_planes(rng, 5, heads, page, D, spread=True)
    cache = to_cache(env, planes)
    slots = rng.integers(-3, 5 * page + 3, n).astype(np.int32)
    got = q4.q4_cache_read(cache, torch.from_numpy(slots).to(dev), out_dtype=getattr(torch, dtype))
    ok = (slots >= 0) & (slots < 5 * page)
    at = np.where(ok, slots, 0)
    for side, g in zip("kv", got):
        w = ref.values(*(planes[f"{side}_{m}"][at // page, :, at % page] for m in ("codes", "scales", "zeros")))
        w[~ok] = 0
        w = w.astype(np.float32)
        if dtype == "bfloat16":
            w = ref.bf16(w)
        assert np.array_equal(g.float().cpu().numpy(), w)


class Batch:
    """Sequences with `new` tokens each and lens[b] keys on random pages."""

    def __init__(self, env, lens, new, heads, G, D, page, seed, spread=False, sharp=1.0, slack=1):
        torch, q4, dev = env
        rng = np.random.default_rng(seed)
        self.lens, new = np.asarray(lens, np.int32), np.asarray(new)
        need = -(-np.maximum(self.lens, 0) // page)
        pages = int(need.sum()) + 2
        self.planes = random_planes(rng, pages, heads, page, D, spread)
        self.table = np.full((len(lens), int(need.max()) + slack if len(lens) else 1), -7, np.int32)
        order, at = rng.permutation(pages), 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(self.offsets[-1])
        self.q = ref.bf16(rng.standard_normal((T, heads * G, D)).astype(np.float32) * sharp)
        self.max_q = int(new.max()) if len(new) else 1
        self.cache = to_cache(env, self.planes)
        d = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        self.dev = (d(self.q).to(torch.bfloat16), self.cache, d(self.table), d(self.lens))
        self.offsets_dev = d(self.offsets)

    def check(self, env, what, causal=True, window=0, scale=None, dtype="bfloat16", tokens=False, **kw):
        torch, q4, dev = env
        kw = dict(q_offsets=None if tokens else self.offsets_dev, max_q=None if tokens else self.max_q, causal=causal,
                  window=window, scale=scale, out_dtype=getattr(torch, dtype), **kw)
        got, lse = q4.q4_cache_attend(*self.dev, return_lse=True, **kw)
        self.plain = q4.q4_cache_attend(*self.dev, **kw)  # (keys of prompts are rounded where no lse is asked for)
        torch.cuda.synchronize()
        out, bound, l, lb, touched = ref.attend(self.q.astype(np.float64), self.planes, self.table, self.lens, self.offsets,
                                                causal, window, scale, dtype == "bfloat16")
        assert touched.all()
        within(got, out, bound, what + " out")
        within(self.plain, out, bound, what + " out alone")
        within(lse, l, lb, what + " lse")
        return got, lse


ATTEND = [  # lens, new tokens, heads, G, D, page
    ([1], [1], 1, 1, 64, 16),
    ([300], [1], 2, 8, 128, 16),
    ([17, 1, 0, 64, 129, 255], [1] * 6, 2, 4, 128, 16),
    ([33, 500, 7, 1000], [1] * 4, 3, 5, 64, 32),
    ([257, 31, 96], [1] * 3, 2, 16, 192, 64),
    ([100, 511, 640], [1] * 3, 1, 7, 256, 128),
    ([90, 40], [1] * 2, 1, 40, 128, 16),
    ([60, 61, 62, 63, 64, 65], [5, 1, 3, 0, 2, 4], 2, 1, 64, 16),
    ([200, 30, 5], [9, 30, 7], 2, 4, 128, 32),
    ([129], [129], 1, 8, 128, 64),
    ([300, 70], [200, 1], 2, 2, 64, 16),
    ([190, 250], [33, 140], 1, 4, 256, 64),
    ([140], [77], 1, 3, 192, 16),
    ([1100], [520], 1, 2, 128, 32),
    ([700, 20, 2000], [130, 20, 1], 2, 3, 64, 16),
    ([777], [300], 1, 1, 256, 128),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
@pytest.mark.parametrize("mode", ["causal", "window", "all"])
def test_attend(env, i, mode):
    lens, new, heads, G, D, page = ATTEND[i]
    b = Batch(env, lens, new, heads, G, D, page, 100 + i, spread=i % 2 == 1, sharp=(0.3, 1.0, 3.0)[i % 3])
    b.check(env, f"{lens} {new} {mode}", causal=mode != "all", window=37 if mode == "window" else 0,
            dtype="float32" if mode == "window" else "bfloat16")
    if mode == "causal" and all(n == 1 for n in new):
        b.check(env, "tokens", tokens=True, scale=0.37)


def test_empty_sequences_and_tokens_of_none(env):
    """Sequences without keys or tokens, tokens before the first and behind the
    last sequence, tokens past max_q: zeros and -infinity where a token sees
    nothing, what was there where it belongs to none."""
    torch, q4, dev = env
    for G, D in ((2, 64), (40, 128)):
        b = Batch(env, [0, 40, 3, 0, 90], [3, 4, 9, 0, 6], 2, G, D, 16, 7)
        T = b.q.shape[0]
        offsets = torch.tensor([2, 3, 7, 16, 16, T - 1], dtype=torch.int32, device=dev)
        for dtype in (torch.bfloat16, torch.float32):
            out = torch.full((T, 2 * G, D), 7.0, dtype=dtype, device=dev)
            lse = torch.full((T, 2 * G), 5.0, device=dev)
            q4.q4_cache_attend(*b.dev, q_offsets=offsets, max_q=8, out=out, lse=lse)
            o, bound, l, lb, touched = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, offsets.cpu().numpy(),
                                                  out_bf16=dtype == torch.bfloat16)
            touched[7 + 8] = False          # the ninth token of its sequence
            kept = torch.from_numpy(~touched).to(dev)
            assert (out[kept] == 7).all() and (lse[kept] == 5).all() and int(kept.sum()) == 4
            at = np.flatnonzero(touched)
            within(out[at], o[at], bound[at], "out")
            within(lse[at], l[at], lb[at], "lse")
            empty = np.isinf(l[at, 0])
            assert empty.sum() >= 7 and (out[at][empty] == 0).all()


def test_pages_of_none_are_hidden(env):
    torch, q4, dev = env
    for new in ([1, 1, 1], [3, 1, 2], [70, 1, 40]):
        b = Batch(env, [100, 77, 200], new, 2, 4, 128, 16, 11)
        rng = np.random.default_rng(3)
        table = b.table.copy()
        for row in table:
            row[rng.integers(0, 4, 2)] = rng.choice([-1, 1 << 30, -2 ** 31, len(b.planes["k_codes"])], 2)
        b.table = table
        b.dev = b.dev[:2] + (torch.from_numpy(table).to(dev), b.dev[3])
        b.check(env, f"hidden {new}")
        b.check(env, f"hidden {new}", causal=False)
    # A sequence all of whose pages are hidden.
    b = Batch(env, [40, 700], [2, 1], 1, 2, 64, 16, 12)
    b.table[:] = -1
    b.dev = b.dev[:2] + (torch.from_numpy(b.table).to(dev), b.dev[3])
    out, lse = b.check(env, "all hidden")
    assert (out == 0).all() and torch.isinf(lse).all()


def _rows_of(b, seq, keys):
    page = b.planes["k_codes"].shape[2]
    return b.table[seq, np.asarray(keys) // page], np.asarray(keys) % page


@pytest.mark.parametrize("new", [[1, 1], [4, 1], [80, 1], [60, 30]])
@pytest.mark.parametrize("slack", [1, 40])
def test_what_a_token_does_not_see_does_not_reach_it(env, new, slack):
    """NaN, infinities and the largest scales in keys behind a token, before its
    window, behind the last key and in the slots of other sequences."""
    torch, q4, dev = env
    heads, G, D, page = 2, 4, 128, 16
    b = Batch(env, [170, 99], new, heads, G, D, page, 21, slack=slack)
    planes = {n: p.copy() for n, p in b.planes.items()}
    used = set()
    for s in range(2):
        ids, at = _rows_of(b, s, np.arange(b.lens[s]))
        used |= set(zip(ids.tolist(), at.tolist()))
    for p in range(planes["k_codes"].shape[0]):
        for i in range(page):
            if (p, i) not in used:
                for n in PLANES:
                    planes[n][p, :, i] = 255 if "codes" in n else np.nan
    # The clean results, then bad keys that the window or the causal mask hides.
    window = 50
    clean, lse0 = b.check(env, "clean", window=window)
    lowest = [int(b.lens[s]) - new[s] - window for s in range(2)]
    bad = {0: [k for k in (0, 5, lowest[0]) if 0 <= k <= lowest[0]], 1: [k for k in (1, lowest[1]) if 0 <= k <= lowest[1]]}
    for s, keys in bad.items():
        for k, v in zip(keys, (np.nan, np.inf, 65504)):
            ids, at = _rows_of(b, s, [k])
            for n in ("k_scales", "v_scales"):
                planes[n][ids[0], :, at[0]] = v
    b.dev = (b.dev[0], to_cache(env, planes)) + b.dev[2:]
    out, lse = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, window=window, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, lse0)
    out = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, window=window)
    assert torch.equal(out, b.plain)


@pytest.mark.parametrize("new", [[1, 1], [5, 1], [80, 1]])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("with_lse", [False, True])
def test_not_finite_values_reach_the_tokens_that_see_them(env, new, side, with_lse):
    """A NaN scale in one block of one key: of a value, the outputs of that block
    in the tokens and heads that see it are NaN; of a key, all of them; the
    others keep their bits."""
    torch, q4, dev = env
    heads, G, D, page = 2, 4, 128, 16
    b = Batch(env, [170, 99], new, heads, G, D, page, 31)
    b.check(env, "clean")

    def attend(cache):
        out = q4.q4_cache_attend(b.dev[0], cache, *b.dev[2:], q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=with_lse)
        return out[0] if with_lse else out

    clean = attend(b.cache)
    for bits in (0x7E00, 0x7C00):
        planes = {n: p.copy() for n, p in b.planes.items()}
        key = 170 - max(1, new[0] // 2)       # about half of the tokens see it
        ids, at = _rows_of(b, 0, [key])
        planes[side + "_scales"].view(np.uint16)[ids[0], 1, at[0], 1] = bits
        planes[side + "_codes"][ids[0], 1, at[0]] = 0x9C
        planes[side + "_zeros"][ids[0], 1, at[0]] = 0
        cache = to_cache(env, planes)
        out = attend(cache).float()
        sees = np.zeros(b.q.shape[0], bool)
        sees[:new[0]] = 170 - new[0] + np.arange(new[0]) >= key
        assert sees.any()
        got = out.cpu().numpy()
        if bits == 0x7E00 or side == "v":
            part = got[sees][:, G:, 64:] if side == "v" else got[sees][:, G:]
            assert np.isnan(part).all()
        keep = np.ones(got.shape, bool)
        keep[np.ix_(sees, range(G, 2 * G), range(64, 128) if side == "v" else range(128))] = False
        if new[0] == 1 or side == "k":
            # (The other block of that key's value is what it was: only codes changed.)
            pass
        if side == "v":
            keep[np.ix_(sees, range(G, 2 * G))] = False
        assert np.array_equal(got[keep], clean.float().cpu().numpy()[keep])


def test_queries_that_are_not_finite_stay_with_their_rows(env):
    torch, q4, dev = env
    for new in ([1, 2], [40, 30]):
        b = Batch(env, [80, 60], new, 2, 4, 64, 16, 41)
        b.check(env, "clean")
        clean = b.plain
        q = b.dev[0].clone()
        q[1, 3, 7] = float("nan")
        q[0, 5, 60] = float("inf")
        out = q4.q4_cache_attend(q, *b.dev[1:], q_offsets=b.offsets_dev, max_q=b.max_q)
        assert torch.isnan(out[1, 3]).all() and torch.isnan(out[0, 5]).all()
        same = torch.ones(out.shape[:2], dtype=torch.bool, device=dev)
        same[1, 3] = same[0, 5] = False
        assert torch.equal(out[same], clean[same])
        # A row of zeros weighs all its keys alike; the largest and smallest queries.
        q = b.dev[0].clone()
        q[0, 0] = 0
        q[0, 1] *= 1e-30
        q[1, 2] *= 2e4
        b.q = q.float().cpu().numpy()
        b.dev = (q,) + b.dev[1:]
        b.check(env, "zero, tiny and large queries")


@pytest.mark.parametrize("new", [[1, 1, 1], [64, 1, 40]])
def test_scales_from_tiny_to_huge(env, new):
    """Scales that grow along the keys (the running exponents move), subnormal
    ones, zeros, and values near the end of fp16."""
    torch, q4, dev = env
    b = Batch(env, [300, 130, 64], new, 2, 2, 128, 16, 51)
    rng = np.random.default_rng(8)
    for s, (lo, hi) in enumerate(((-22, 3), (3, -20), (-24, -24))):
        n = int(b.lens[s])
        ids, at = _rows_of(b, s, np.arange(n))
        e = np.linspace(lo, hi, n)[:, None, None] + rng.integers(-1, 2, (n, 2, 2))
        b.planes["v_scales"][ids, :, at] = (2.0 ** np.clip(e, -24, 15) * rng.uniform(1, 1.9, e.shape)).astype(np.float16)
        b.planes["k_scales"][ids, :, at] = (2.0 ** np.clip(-np.abs(e) / 2, -24, 0)).astype(np.float16)
    b.planes["v_scales"][b.table[0, 0], 0, 3] = 0
    b.dev = (b.dev[0], to_cache(env, b.planes)) + b.dev[2:]
    b.check(env, "scales", dtype="float32")
    ids, at = _rows_of(b, 0, np.arange(290, 300))
    b.planes["v_scales"][ids, :, at] = 4300.0      # times up to 15: past 64000
    b.dev = (b.dev[0], to_cache(env, b.planes)) + b.dev[2:]
    b.check(env, "large values", dtype="float32")


def test_one_page_for_many_and_the_same_page_twice(env):
    """A shared prefix: sequences whose tables name the same pages, one page in
    several places of a table."""
    torch, q4, dev = env
    b = Batch(env, [200, 150, 90], [1, 40, 3], 2, 3, 64, 16, 61)
    b.table[1, :5] = b.table[0, :5]
    b.table[2, :5] = b.table[0, 2]
    b.dev = b.dev[:2] + (torch.from_numpy(b.table).to(dev), b.dev[3])
    b.check(env, "shared pages")


def test_long_context_and_many_sequences(env):
    """More tiles than waves, more sequences than a workgroup has threads."""
    torch, q4, dev = env
    rng = np.random.default_rng(71)
    lens = rng.integers(0, 40, 700)
    lens[::97] = 400
    b = Batch(env, lens, rng.integers(0, 3, 700), 1, 2, 64, 16, 72, slack=120)
    b.check(env, "700 sequences")
    b = Batch(env, [9000, 5, 2111], [1, 1, 1], 3, 3, 64, 32, 73, sharp=2.0)
    b.check(env, "long")
    b = Batch(env, [2500, 400], [150, 90], 1, 4, 64, 32, 74)
    b.check(env, "parts", dtype="float32")


def test_strided_queries_and_given_outputs(env):
    torch, q4, dev = env
    b = Batch(env, [50, 70], [2, 40], 2, 4, 64, 16, 81)
    T = b.q.shape[0]
    wide = torch.full((T, 12, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 2:10] = b.dev[0]
    first, _ = b.check(env, "dense")
    out = torch.empty((T, 8, 64), dtype=torch.bfloat16, device=dev)
    need = q4.q4_cache_attend_ws_bytes(T, 8, 2, 64, 2, b.max_q)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
    got = q4.q4_cache_attend(wide[:, 2:10], *b.dev[1:], q_offsets=b.offsets_dev, max_q=b.max_q, out=out, workspace=ws,
                             lse=torch.empty((T, 8), device=dev))
    assert got is out and torch.equal(out, first)
    with pytest.raises(q4.Q4Error):
        q4.q4_cache_attend(wide[:, 2:10], *b.dev[1:], q_offsets=b.offsets_dev, max_q=b.max_q, out=out, workspace=ws[:-16])


def test_the_same_bits_on_every_call(env):
    torch, q4, dev = env
    for new, lens in (([1, 1], [5000, 300]), ([200, 60], [3000, 60])):
        b = Batch(env, lens, new, 2, 4, 128, 16, 91)
        run = lambda: q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, out_dtype=torch.float32, return_lse=True)  # noqa: E731
        o, l = run()
        for _ in range(3):
            o2, l2 = run()
            assert torch.equal(o, o2) and torch.equal(l, l2)
