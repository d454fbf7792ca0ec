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
