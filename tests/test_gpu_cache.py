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
        within(q, w, (2.0 ** -8 + 2.0 ** -24) * np.abs(w) + 1e-37, "rotated q")
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
                                                  (300, 2, 256, 128, "bfloat16")])
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
        got, lse = q4.q4_cache_attend(*self.dev, q_offsets=None if tokens else self.offsets_dev,
                                      max_q=None if tokens else self.max_q, causal=causal, window=window, scale=scale,
                                      out_dtype=getattr(torch, dtype), return_lse=True, **kw)
        torch.cuda.synchronize()
        out, bound, l, lb, touched = ref.attend(self.q.astype(np.float64), self.planes, self.table, self.lens, self.offsets,
                                                causal, window, scale, dtype == "bfloat16")
        assert touched.all()
        within(got, out, bound, what + " out")
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
