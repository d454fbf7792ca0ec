"""The cache's binding where it makes or leaves out planes (bit_weight_gemv_amd/cache.py),
on CPU tensors: nothing is launched."""
import pytest


@pytest.mark.parametrize("D", [65, 66, 127, 129, 0, -64, 32])
def test_a_new_cache_has_the_dimensions_asked_for_or_none(D):
    pytest.importorskip("torch")
    import bit_weight_gemv_amd as q4
    with pytest.raises(ValueError):
        q4.q4_cache_new(2, 2, 16, D, "cpu")
    assert q4.q4_cache_new(2, 2, 16, 192, "cpu").D == 192


def test_read_refuses_outputs_of_what_it_does_not_read():
    torch = pytest.importorskip("torch")
    import bit_weight_gemv_amd as q4
    c = q4.q4_cache_new(2, 2, 16, 64, "cpu")
    slots, out = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64)
    for kw in (dict(keys=False, values=False), dict(keys=False, k_out=out), dict(values=False, v_out=out)):
        with pytest.raises(ValueError):
            q4.q4_cache_read(c, slots, **kw)
