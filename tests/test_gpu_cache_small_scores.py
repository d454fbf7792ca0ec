"""Attention where the scores are small or zero: query rows of zeros (padding),
keys whose scales are zero or tiny, and a small `scale`.  The weights are then
all but equal, and out is the mean of the seen values.  Bounds:
tests/cache_reference.py."""
import numpy as np
import pytest

from test_gpu_cache import Batch, env, to_cache  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [  # lens, new tokens, heads, G, D
    ([120, 90, 77], [80, 70, 77], 1, 1, 128),      # prompts: more than 64 rows a key head
    ([130, 20, 50], [40, 20, 33], 2, 4, 64),
    ([90, 64, 70], [50, 40, 35], 1, 2, 256),       # (more than 32 for D > 128)
    ([60, 50, 40], [40, 33, 9], 1, 3, 192),
    ([700, 1400, 90], [9, 1, 5], 2, 3, 128),       # drafts and tokens
    ([300, 200, 100], [1, 1, 1], 2, 8, 64),
    ([3000, 50, 40], [1, 2, 1], 1, 5, 256),
]


def batch(env, i, key_scales):
    """key_scales: of each sequence, a scale or a choice of them."""
    lens, new, heads, G, D = SHAPES[i]
    rng = np.random.default_rng(500 + i)
    b = Batch(env, lens, new, heads, G, D, 16, 400 + i, slack=80 if i > 3 else 1)
    for s, choice in enumerate(key_scales):
        pages = b.table[s, :-(-lens[s] // 16)]
        shape = b.planes["k_scales"][pages].shape
        b.planes["k_scales"][pages] = rng.choice(np.asarray(choice, np.float16).reshape(-1), shape)
    b.q[::2] = 0                     # every other token is padding
    b.q[1::4, ::2] *= 2.0 ** -120    # tiny rows, down to bf16's subnormals
    b.q[1::4, 1::2] *= 2.0 ** -60
    torch, q4, dev = env
    q = torch.from_numpy(b.q).to(dev).to(torch.bfloat16)
    b.q = q.float().cpu().numpy()
    b.dev = (q, to_cache(env, b.planes)) + b.dev[2:]
    return b


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-30, 1e-12, 0.01, None, 1.0])
@pytest.mark.parametrize("window", [0, 21])
def test_rows_of_zeros_take_the_mean_of_what_they_see(env, i, scale, window):
    for what, scales in (("zero and tiny keys", (0.0, 2.0 ** -14, 2.0 ** -20)),
                         ("mixed keys", ([0.0, 2.0 ** -14], [2.0 ** -24, 0.25], [0.0, 0.25])),
                         ("keys", (0.25, 0.25, 0.0))):
        b = batch(env, i, scales)
        out, lse = b.check(env, f"{what}, scale {scale}, window {window}", scale=scale, window=window, dtype="float32")
        for x in (out, lse, b.plain):
            assert x.isfinite().all()


@pytest.mark.parametrize("new", [[70, 1], [3, 1]])
def test_a_warm_up_over_zeroed_buffers(env, new):
    """Queries and cache all zeros: zeros out, lse the logarithm of the keys."""
    torch, q4, dev = env
    cache = q4.KVCache(*(torch.zeros((8, 2, 16, n), dtype=t, device=dev) for _ in range(2)
                         for n, t in ((64, torch.uint8), (2, torch.float16), (2, torch.float16))))
    T = sum(new)
    i32 = dict(dtype=torch.int32, device=dev)
    offsets = torch.tensor([0, new[0], T], **i32)
    args = (torch.zeros(T, 4, 128, dtype=torch.bfloat16, device=dev), cache, torch.full((2, 5), 3, **i32),
            torch.tensor([new[0], 9], **i32), offsets, max(new))
    out, lse = q4.q4_cache_attend(*args, return_lse=True)
    assert (out == 0).all() and (q4.q4_cache_attend(*args) == 0).all()
    keys = torch.cat([torch.arange(1, new[0] + 1), torch.tensor([9])]).double().log()[:, None].expand(T, 4)
    # The logarithm of up to 70 weights of 2^33, within a step of 2^-18 (times ln 2).
    assert (lse.cpu().double() - keys).abs().max() <= 2.0 ** -18


@pytest.mark.parametrize("new", [[80, 1], [3, 1], [1, 1]])
def test_rows_of_large_queries_over_keys_of_zeros(env, new):
    """The largest bf16 values: scores of zero stay zero."""
    torch, q4, dev = env
    b = Batch(env, [100, 70], new, 2, 2, 128, 16, 77)
    b.planes["k_scales"][:] = 0
    q = b.dev[0].clone()
    q[0] = 3.0e38
    q[1, 1] = -1e37
    b.q = q.float().cpu().numpy()
    b.dev = (q, to_cache(env, b.planes)) + b.dev[2:]
    for scale in (None, 1.0, 1e30):
        b.check(env, f"large queries, scale {scale}", scale=scale, dtype="float32")
