"""The cache's calls together, as a serving step makes them (q4_cache.h): behind
and before packed projections, captured in graphs, on other streams, and on
caches past 32-bit offsets."""
import numpy as np
import pytest

import cache_reference as ref
from test_gpu_cache import PLANES, Batch, env, of_cache, random_planes, to_cache, within  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_layer_of_prompt_and_tokens(env):
    """q, k and v from a packed projection; a prompt in two chunks, then tokens
    one by one, two sequences; the output through a packed projection."""
    torch, q4, dev = env
    rng = np.random.default_rng(1)
    Hq, H, D, page, hidden, pages = 6, 2, 64, 16, 256, 12
    W = torch.from_numpy(rng.standard_normal(((Hq + 2 * H) * D, hidden)).astype(np.float32) * 0.06).to(dev)
    codes, scales, _ = q4.q4_pack(W)
    Wo = torch.from_numpy(rng.standard_normal((hidden, Hq * D)).astype(np.float32) * 0.05).to(dev)
    oc, os_, _ = q4.q4_pack(Wo)
    cache = to_cache(env, {n: p for n, p in random_planes(rng, pages, H, page, D).items()})
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).to(dev)
    order = rng.permutation(pages)
    table = np.stack([order[:6], order[6:]]).astype(np.int32)
    tabled = torch.from_numpy(table).to(dev)
    lens = np.zeros(2, np.int32)
    planes = of_cache(cache)
    for step, new in enumerate(([30, 17], [25, 1], [1, 1], [1, 1], [0, 1], [1, 4])):
        T = sum(new)
        offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = np.concatenate([lens[b] + np.arange(n) for b, n in enumerate(new)]).astype(np.int32)
        seq = np.repeat([0, 1], new)
        slots = (table[seq, pos // page] * page + pos % page).astype(np.int32)
        lens = lens + np.asarray(new, np.int32)
        X = torch.from_numpy(ref.bf16(rng.standard_normal((T, hidden)))).to(dev).to(torch.bfloat16)
        qkv = torch.cat([q4.q4_gemm_smalln(codes, scales, x) for x in X.split(32)]).view(T, Hq + 2 * H, D)
        q = q4.q4_cache_append(cache, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], torch.from_numpy(slots).to(dev),
                               torch.from_numpy(pos).to(dev), freq, q=qkv[:, :Hq])
        out = q4.q4_cache_attend(q, cache, tabled, torch.from_numpy(lens).to(dev), torch.from_numpy(offsets).to(dev), max(new))
        y = torch.cat([q4.q4_gemm_smalln(oc, os_, x) for x in out.view(T, Hq * D).split(32)])
        # The same in 64 bits, from the projection's output.
        x = qkv.cpu().numpy().astype(np.float64)
        f = freq.cpu().numpy()
        for side, rows in (("k", ref.rotate(x[:, Hq:Hq + H], pos, f, False, 1.0)), ("v", x[:, Hq + H:])):
            for name, r in zip(("codes", "scales", "zeros"), ref.pack(rows)):
                planes[f"{side}_{name}"][slots // page, :, slots % page] = r
        got = of_cache(cache)
        for n in PLANES:
            assert np.array_equal(got[n], planes[n]), (step, n)
        want, bound, _, _, _ = ref.attend(q.float().cpu().numpy().astype(np.float64), planes, table, lens, offsets)
        within(out, want, bound, f"step {step}")
        o = out.float().cpu().numpy().astype(np.float64).reshape(T, -1)
        w = Wo.cpu().numpy().astype(np.float64)
        # A packed weight is off by half a step of its block's 16 levels: 0.16 of its scale.
        err = np.abs(y.cpu().numpy() - o @ w.T)
        s = np.repeat(os_.float().cpu().numpy(), 64, axis=1)
        assert (err <= (np.abs(o) @ (0.16 * s).T) + 1e-3 * (np.abs(o) @ np.abs(w).T) + 1e-5).all()


def test_captured_steps_as_sequences_grow(env):
    """A step captured once: append, attend, read; replayed as lengths, slots and
    positions change in place, with eager calls between; a second graph shares
    the workspace."""
    torch, q4, dev = env
    rng = np.random.default_rng(2)
    for lens0, qh, D, new in (([700, 90, 33], 8, 128, 1), ([60, 5, 200], 4, 64, 30), ([3000, 1, 1500], 2, 64, 1)):
        b = Batch(env, np.asarray(lens0) + 8 * new, [new] * 3, 2, qh // 2, D, 16, 5)
        T = 3 * new
        lens = torch.tensor(lens0, dtype=torch.int32, device=dev)
        kv = torch.randn(T, 4, D, device=dev)
        slots = torch.zeros(T, dtype=torch.int32, device=dev)
        pos = torch.zeros(T, dtype=torch.int32, device=dev)
        freq = torch.from_numpy((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).to(dev)
        q = torch.randn(T, qh, D, device=dev)
        need = q4.q4_cache_attend_ws_bytes(T, qh, 2, D, 3, new)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        table, offsets = b.dev[2], b.offsets_dev

        def advance():
            for s in range(3):
                p = int(lens[s]) + torch.arange(new, device=dev)
                pos[s * new:(s + 1) * new] = p.int()
                slots[s * new:(s + 1) * new] = (table[s][p // 16] * 16 + p % 16).int()
            lens.add_(new)
            kv.normal_()
            q.normal_()

        def step(cache, qo, out, lse, k, v):
            q4.q4_cache_append(cache, kv[:, :2], kv[:, 2:], slots, pos, freq, q=q, q_out=qo)
            q4.q4_cache_attend(qo, cache, table, lens, offsets, new, out=out, lse=lse, workspace=ws)
            q4.q4_cache_read(cache, slots, k_out=k, v_out=v)

        def outputs():
            bf = dict(dtype=torch.bfloat16, device=dev)
            return (torch.zeros(T, qh, D, **bf), torch.zeros(T, qh, D, **bf), torch.zeros(T, qh, device=dev),
                    torch.zeros(T, 2, D, **bf), torch.zeros(T, 2, D, **bf))

        eager, captured, second = outputs(), outputs(), outputs()
        other = to_cache(env, b.planes)
        advance()
        step(b.cache, *eager)
        step(other, *captured)
        torch.cuda.synchronize()
        graphs = []
        for target in (captured, second):
            g = torch.cuda.CUDAGraph()
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                with torch.cuda.graph(g, stream=st):
                    step(other, *target)
            graphs.append(g)
        torch.cuda.synchronize()
        for rep in range(4):
            advance()
            torch.cuda.synchronize()
            step(b.cache, *eager)
            torch.cuda.synchronize()
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for e, c, s in zip(eager, captured, second):
                assert torch.equal(e, c) and torch.equal(e, s), rep
            for n in PLANES:
                assert torch.equal(getattr(b.cache, n), getattr(other, n))


def test_calls_on_two_streams_at_once(env):
    torch, q4, dev = env
    a = Batch(env, [3000, 200], [1, 1], 2, 4, 128, 16, 6)
    c = Batch(env, [900, 400], [200, 100], 2, 2, 64, 16, 7)
    a.check(env, "a")
    c.check(env, "c")
    want_a, want_c = a.plain, c.plain
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((q4.q4_cache_attend(*a.dev, q_offsets=a.offsets_dev, max_q=1, stream=s1),
                    q4.q4_cache_attend(*c.dev, q_offsets=c.offsets_dev, max_q=c.max_q, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want_a) and torch.equal(y, want_c)


def test_caches_past_32_bits(env):
    """Pages behind 4 GiB of codes (and 2^31 values): the rows that are written,
    read and seen are those of the same pages in a small cache."""
    torch, q4, dev = env
    if torch.cuda.get_device_properties(dev).total_memory < 40 << 30:
        pytest.skip("needs 40 GiB")
    heads, page, D = 8, 64, 256
    pages = (1 << 32) // (heads * page * D // 2) + 40
    big = q4.q4_cache_new(pages, heads, page, D, dev)
    assert big.k_codes.numel() > 1 << 32
    for new in ([1, 2], [40, 30]):
        b = Batch(env, [900, 300], new, heads, 2, D, page, 8)
        small = b.planes["k_codes"].shape[0]
        at = pages - 1 - torch.arange(small, device=dev)   # the last pages, in reverse
        assert 0 <= int(at.min()) and int(at.max()) < pages
        for n in PLANES:
            getattr(big, n)[at] = getattr(b.cache, n)
        table = torch.where(b.dev[2] < 0, b.dev[2], at.int()[b.dev[2].clamp(min=0).long()])
        want, lse = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=True)
        got, lse2 = q4.q4_cache_attend(b.dev[0], big, table, b.dev[3], q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=True)
        assert torch.equal(want, got) and torch.equal(lse, lse2)
    k = torch.randn(3, heads, D, device=dev)
    top = torch.tensor([pages * page - 1, pages * page - 70, 5], dtype=torch.int32, device=dev)
    few = q4.q4_cache_new(1, heads, page, D, dev)
    here = torch.tensor([1, 2, 3], dtype=torch.int32, device=dev)
    q4.q4_cache_append(big, k, -k, top)
    q4.q4_cache_append(few, k, -k, here)
    for x, y in zip(q4.q4_cache_read(big, top), q4.q4_cache_read(few, here)):
        assert torch.equal(x, y)


def test_lengths_past_the_table_are_held_to_it(env):
    torch, q4, dev = env
    b = Batch(env, [64, 48], [1, 1], 2, 2, 64, 16, 10, slack=0)
    long = torch.tensor([64, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    b.lens = np.asarray([64, b.table.shape[1] * 16], np.int32)
    b.table[1, 3:] = b.table[1, 0]
    b.dev = b.dev[:2] + (torch.from_numpy(b.table).to(dev), long)
    b.check(env, "held")
    neg = torch.tensor([-5, -2 ** 31], dtype=torch.int32, device=dev)
    out, lse = q4.q4_cache_attend(b.dev[0], b.cache, b.dev[2], neg, return_lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_offsets_out_of_order_stay_in_bounds(env):
    """Offsets against the contract: the outputs are unspecified, the accesses
    are not (the guard rows keep what they held)."""
    torch, q4, dev = env
    b = Batch(env, [64, 48, 200], [2, 30, 1], 2, 4, 64, 16, 11)
    T = b.q.shape[0]
    guard = torch.full((T + 8, 8, 64), 3.0, dtype=torch.bfloat16, device=dev)
    for bad in ([0, 40, 2, T], [-5, T + 900, T, 1], [2 ** 31 - 1, 0, -2 ** 31, 2 ** 31 - 1], [T, 5, 3, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device=dev)
        q4.q4_cache_attend(*b.dev, q_offsets=off, max_q=T, out=guard[:T])
        torch.cuda.synchronize()
        assert (guard[T:] == 3).all()


def test_no_tokens_no_sequences_no_pages(env):
    torch, q4, dev = env
    c = q4.q4_cache_new(0, 2, 16, 64, dev)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    lens = torch.tensor([5, 0, 9], **i32)
    out, lse = q4.q4_cache_attend(q, c, torch.zeros(3, 2, **i32), lens, return_lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()
    out = q4.q4_cache_attend(q, c, torch.zeros(3, 0, **i32), lens)
    assert (out == 0).all()
    assert q4.q4_cache_attend(q[:0], c, torch.zeros(0, 2, **i32), lens[:0]).shape == (0, 4, 64)
    k = torch.zeros(3, 2, 64, device=dev)
    q4.q4_cache_append(c, k, k, torch.tensor([0, 1, -1], **i32))
    assert q4.q4_cache_append(c, k[:0], k[:0], torch.zeros(0, **i32), q=k[:0]).shape == (0, 2, 64)
    r, _ = q4.q4_cache_read(c, torch.tensor([0, 7], **i32))
    assert (r == 0).all()
