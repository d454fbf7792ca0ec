"""Calls of the 4-bit cache at the borders of its contract: tables far wider
than the sequences, windows that reach past the first key, slots given twice,
single tokens out of larger tensors.  Bounds: tests/cache_reference.py."""
import numpy as np
import pytest

import cache_reference as ref
from test_gpu_cache import Batch, PLANES, env, of_cache, random_planes, to_cache  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new,heads,G,D,window,slack", [
    ([3001], [40], 2, 2, 64, 0, 3000),           # keys in parts, whatever the table holds
    ([2600, 300], [150, 70], 2, 2, 128, 0, 999),
    ([3001], [70], 1, 3, 128, 900, 5),           # parts of a window
    ([2000, 1500, 9], [90, 66, 1], 1, 1, 256, 700, 200),
])
def test_parts_follow_what_is_seen(env, lens, new, heads, G, D, window, slack):
    b = Batch(env, lens, new, heads, G, D, 16, 200 + D + slack, slack=slack)
    b.check(env, f"{lens} {new} window {window} slack {slack}", window=window, dtype="float32")


@pytest.mark.parametrize("new", [[1, 1, 1], [9, 3, 50], [90, 1, 400]])
def test_windows_past_the_first_key_hide_nothing(env, new):
    """Also of tokens that stand before the first key (more tokens than keys)."""
    torch, q4, dev = env
    b = Batch(env, [200, 1, 300], new, 2, 2, 64, 32, 31)
    run = lambda w: q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, window=w, return_lse=True)  # noqa: E731
    out, lse = b.check(env, "none")
    for w in (b.table.shape[1] * 32 + 1, 1 << 30, 2 ** 31 - 1):
        o, l = run(w)
        assert torch.equal(o, out) and torch.equal(l, lse)
    b.check(env, "as long as the table", window=b.table.shape[1] * 32)


def test_a_slot_given_twice_stays_within_its_rows(env):
    torch, q4, dev = env
    rng = np.random.default_rng(5)
    heads, D, page, T = 3, 128, 16, 90
    planes = random_planes(rng, 8, heads, page, D)
    cache = to_cache(env, planes)
    x = [ref.bf16(rng.standard_normal((T, heads, D)).astype(np.float32)) for _ in range(2)]
    slots = rng.permutation(8 * page)[:T].astype(np.int32)
    twice = slots[7]
    slots[[20, 21, 64]] = twice
    d = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    q4.q4_cache_append(cache, d(x[0]).to(torch.bfloat16), d(x[1]).to(torch.bfloat16), d(slots))
    got = of_cache(cache)
    for side, v in zip("kv", x):
        want = {m: planes[f"{side}_{m}"].copy() for m in ("codes", "scales", "zeros")}
        for m, p in zip(("codes", "scales", "zeros"), ref.pack(v)):
            want[m][slots // page, :, slots % page] = p
        for m in want:
            g, w = got[f"{side}_{m}"], want[m]
            other = np.ones((8, page), bool)
            other[twice // page, twice % page] = False
            g, w = (np.moveaxis(a, 2, 1)[other] for a in (g, w))
            assert np.array_equal(g.view(np.uint8), w.view(np.uint8)), (side, m)


def test_one_token_of_a_larger_tensor(env):
    """The distance to the next token does not count where there is none."""
    torch, q4, dev = env
    rng = np.random.default_rng(6)
    heads, D, page = 2, 64, 16
    x = torch.from_numpy(rng.standard_normal((1, heads * D + 3)).astype(np.float32)).to(dev).to(torch.bfloat16)
    part = x.as_strided((1, heads, D), (heads * D + 3, D, 1))
    assert part.stride(0) % 8 != 0
    slot = torch.tensor([17], dtype=torch.int32, device=dev)
    caches = [to_cache(env, random_planes(np.random.default_rng(7), 2, heads, page, D)) for _ in range(2)]
    for cache, t in zip(caches, (part, part.contiguous())):
        q4.q4_cache_append(cache, t, t, slot)
    a, b = (of_cache(c) for c in caches)
    assert all(np.array_equal(a[n].view(np.uint8), b[n].view(np.uint8)) for n in PLANES)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([18], dtype=torch.int32, device=dev)
    out = [q4.q4_cache_attend(t, caches[0], table, lens) for t in (part, part.contiguous())]
    assert torch.equal(*out)


@pytest.mark.parametrize("lens,new,G,D", [([700, 333], [300, 90], 4, 128), ([500], [200], 1, 64), ([400], [66], 5, 192),
                                          ([300, 900], [130, 100], 2, 256), ([2000, 64], [1, 5], 7, 128)])
def test_lse_has_the_precision_of_its_type(env, lens, new, G, D):
    """lse is fp32, and so are its scores: keys enter the products exactly.  A
    score's D products and ND scaled sums are added in fp32, every step rounded
    by 2^-24 of at most sum |q| |code - zero| scale, doubled where zero points
    are subtracted behind (30 for 15), with 2^-24 for each product that a
    matrix core aligns: 2 (2 D + 16) 2^-24 of 30 sum |q| scale bounds every
    score; the sum of the weights adds (keys + 16) 2^-24, the exponent and the
    logarithm 2^-22 of the largest score and 1.  Of independent roundings the
    2-norm over all rows stays below half of 2e-5 of the norm of lse."""
    torch, q4, dev = env
    b = Batch(env, lens, new, 2, G, D, 16, 300 + D, sharp=2.0)
    _, lse = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=True)
    got = lse.cpu().numpy().astype(np.float64)
    _, _, want, _, _ = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, b.offsets)
    assert np.isfinite(want).all()
    # The largest block sums of |q| times scales 0.5 at most.
    most = 30 * 0.5 * np.abs(b.q.astype(np.float64)).sum(-1) * D ** -0.5
    bound = 2 * (2 * D + 16) * 2.0 ** -24 * most + (max(lens) + 16) * 2.0 ** -24 + 2.0 ** -22 * (most + 1)
    assert (np.abs(got - want) <= bound).all()
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    print(f"{lens} {new} D {D}: lse off by {rel:.2g} (2-norm), {np.abs(got - want).max():.2g} at most", flush=True)
    assert rel < 1e-5
