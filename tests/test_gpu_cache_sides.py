"""q4_cache_read of one side alone: the same rows, and nothing in the other's place."""
import numpy as np
import pytest

from test_gpu_cache import env, random_planes, to_cache  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads,D", [(5, 2, 64), (900, 3, 192), (6000, 8, 128)])
def test_keys_alone_and_values_alone(env, n, heads, D):
    torch, q4, dev = env
    rng = np.random.default_rng(n)
    cache = to_cache(env, random_planes(rng, 6, heads, 32, D))
    slots = torch.from_numpy(rng.integers(-2, 6 * 32 + 2, n).astype(np.int32)).to(dev)
    for dtype in (torch.bfloat16, torch.float32):
        k, v = q4.q4_cache_read(cache, slots, out_dtype=dtype)
        k1, none = q4.q4_cache_read(cache, slots, out_dtype=dtype, values=False)
        assert none is None and torch.equal(k, k1)
        given = torch.empty_like(v)
        none, v1 = q4.q4_cache_read(cache, slots, v_out=given, keys=False)
        assert none is None and v1 is given and torch.equal(v, v1)
