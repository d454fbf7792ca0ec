"""Limits of the experts' and the adapters' entry points without a GPU: what is
within them is not refused.  Null pointers end each call behind the check of
its shape."""
from test_boundary_experts_lora import P, _combine, _grouped, q4  # noqa: F401


def test_combine_limit_counts_the_workgroups_that_run(q4):  # noqa: F811
    """Rows of whole 16-byte pieces take 2048 columns a workgroup, others 256;
    a launch holds fewer than 2^24 workgroups of 256."""
    none = [None] * 4
    for T, M in ((1 << 17, 1 << 15), (1 << 22, 6144), ((1 << 21) - 1, 16384), ((1 << 16) - 1, 65535)):
        assert _combine(q4, T=T, M=M, p=none) == q4.Q4_ERR_NULL, (T, M)
    for T, M in ((1 << 21, 16384), (1 << 16, 65535), (1 << 22, 6145)):
        assert _combine(q4, T=T, M=M, p=none) == q4.Q4_ERR_SHAPE, (T, M)


def test_grouped_limit_of_the_launch_that_converts_activations(q4):  # noqa: F811
    """A wave of that launch takes 256 k of two rows: 2^24 workgroups of four
    waves hold fewer than 2^26 such pairs."""
    kw = dict(E=1024, M=11, T=5, up=True, p=[None, None, P(2), None, None, None, None, None])
    assert _grouped(q4, K=131072, R=(1 << 18) - 2, **kw) == q4.Q4_ERR_NULL
    assert _grouped(q4, K=131072, R=1 << 18, **kw) == q4.Q4_ERR_SHAPE
    assert _grouped(q4, K=2048, R=923858, **kw) == q4.Q4_ERR_NULL
