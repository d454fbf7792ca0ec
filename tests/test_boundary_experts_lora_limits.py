"""Limits of the experts' and the adapters' entry points without a GPU: what is
within them is not refused.  Null pointers end each call behind the check of
its shape."""
from test_boundary_experts_lora import _combine, q4  # noqa: F401


def test_combine_limit_counts_the_workgroups_that_run(q4):  # noqa: F811
    """Rows of whole 16-byte pieces take 2048 columns a workgroup, others 256;
    a launch holds fewer than 2^24 workgroups of 256."""
    none = [None] * 4
    for T, M in ((1 << 17, 1 << 15), (1 << 22, 6144), ((1 << 21) - 1, 16384), ((1 << 16) - 1, 65535)):
        assert _combine(q4, T=T, M=M, p=none) == q4.Q4_ERR_NULL, (T, M)
    for T, M in ((1 << 21, 16384), (1 << 16, 65535), (1 << 22, 6145)):
        assert _combine(q4, T=T, M=M, p=none) == q4.Q4_ERR_SHAPE, (T, M)
