"""What include/q4_cache.h says of large scores, of queries that are not finite,
of scales that no packing writes, and of a NaN value's extent."""
import numpy as np
import pytest

import cache_reference as ref
from test_gpu_cache import Batch, _rows_of, env, to_cache, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new,heads,G,D,slack", [([300, 90], [1, 1], 2, 4, 128, 1), ([3000, 90], [3, 1], 1, 2, 64, 1),
                                                      ([200, 130], [80, 60], 1, 2, 128, 1), ([400], [60], 1, 1, 256, 1)])
@pytest.mark.parametrize("lse", [False, True])
def test_scores_up_to_2_to_24(env, lens, new, heads, G, D, slack, lse):
    """Scores up to 2^24 in magnitude: the weight is with the largest.  A score is
    off by 2^-11 of D products at most (keys rounded to fp16); rows whose second
    largest is further away than that have the largest one's value."""
    torch, q4, dev = env
    b = Batch(env, lens, new, heads, G, D, 16, 3, slack=slack)
    x = b.q.astype(np.float64)
    K = ref.values(*(b.planes["k_" + n] for n in ("codes", "scales", "zeros")))
    V = ref.values(*(b.planes["v_" + n] for n in ("codes", "scales", "zeros")))
    most = max(np.abs(np.einsum("phid,thd->pith", K[:, np.arange(heads * G) // G], x)).max(), 1)
    scale = float(np.float32(0.9 * 2.0 ** 24 / most))
    out = q4.q4_cache_attend(*b.dev, q_offsets=b.offsets_dev, max_q=b.max_q, scale=scale, out_dtype=torch.float32, return_lse=lse)
    out = (out[0] if lse else out).cpu().numpy()
    assert np.isfinite(out).all()
    clear = 0
    for s in range(len(lens)):
        for j in range(new[s]):
            ids, at = _rows_of(b, s, np.arange(lens[s] - new[s] + j + 1))
            for h in range(heads * G):
                k, v, q = K[ids, h // G, at], V[ids, h // G, at], x[b.offsets[s] + j, h]
                score = scale * (k @ q)
                err = 2 * 2.0 ** -10 * scale * (np.abs(k) @ np.abs(q)).max() + 64
                best = np.argsort(score)[-2:]
                if len(best) == 1 or score[best[1]] - score[best[0]] > err:
                    clear += 1
                    assert np.abs(out[b.offsets[s] + j, h] - v[best[-1]]).max() <= 2.0 ** -9 * np.abs(v[best[-1]]).max()
    print("rows with one key far ahead:", clear, "of", out.shape[0] * out.shape[1])
    assert 2 * clear > out.shape[0] * out.shape[1]


@pytest.mark.parametrize("new", [[1, 1], [5, 2], [80, 60]])
def test_rows_of_q_that_are_not_finite(env, new):
    """NaN (or the formula's value) where the row sees a key, zeros and -infinity
    where it sees none; the other rows keep their bits."""
    torch, q4, dev = env
    b = Batch(env, [100, 70], new, 2, 2, 128, 16, 8)
    kw = dict(q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=True)
    clean = q4.q4_cache_attend(*b.dev, **kw)
    q = b.dev[0].clone()
    q[0, 1, 5], q[1, 2, 127] = float("nan"), float("-inf")
    got = q4.q4_cache_attend(q, *b.dev[1:], **kw)
    assert torch.isnan(got[0][0, 1]).all() and torch.isnan(got[1][0, 1])
    same = torch.ones(q.shape[:2], dtype=torch.bool, device=dev)
    same[0, 1] = same[1, 2] = False
    for g, c in zip(got, clean):
        assert torch.equal(g[same], c[same])
    out, lse = q4.q4_cache_attend(q, *b.dev[1:3], torch.zeros_like(b.dev[3]), **kw)
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("new", [[1, 1], [5, 2], [80, 60]])
@pytest.mark.parametrize("bits", [0x8000, 0x9400, 0x7C00, 0xFC00])
def test_scales_that_no_packing_writes_stay_with_those_that_see_them(env, new, bits):
    """-0, negative and infinite scales: unspecified for the rows that see the key,
    and no more than that.  The others are within their bound, not the same
    to the bit: the rows of a tile take up a new maximum m together, and a score
    of the key may have them do so at another key.  Weights are 2^(s - m) then for
    another m, each still rounded once by 2^-11, and the sums are divided by
    theirs: every term of the bound holds for any m."""
    torch, q4, dev = env
    b = Batch(env, [170, 99], new, 2, 4, 128, 16, 9)
    kw = dict(q_offsets=b.offsets_dev, max_q=b.max_q)
    want, bound, _, _, _ = ref.attend(b.q.astype(np.float64), b.planes, b.table, b.lens, b.offsets)
    for with_lse in (False, True):
        for side in "kv":
            planes = {n: p.copy() for n, p in b.planes.items()}
            key = 170 - max(1, new[0] // 2)
            ids, at = _rows_of(b, 0, [key])
            planes[side + "_scales"].view(np.uint16)[ids[0], 1, at[0], :] = bits
            out = q4.q4_cache_attend(b.dev[0], to_cache(env, planes), *b.dev[2:], return_lse=with_lse, **kw)
            out = out[0] if with_lse else out
            blind = np.ones(out.shape[:2], bool)
            blind[:new[0], 4:] = (170 - new[0] + np.arange(new[0]) < key)[:, None]
            within(out[torch.from_numpy(blind).to(dev)], want[blind], bound[blind], f"{side}, scale bits {bits:#x}, lse {with_lse}")


@pytest.mark.parametrize("new", [[1, 1], [5, 1], [80, 1]])
@pytest.mark.parametrize("with_lse", [False, True])
def test_a_value_that_is_not_finite_fills_its_block_alone(env, new, with_lse):
    """A NaN value scale in the second block of one key: that block's outputs are
    NaN in the tokens and heads that see the key; their other block keeps its
    bits, as do all others."""
    torch, q4, dev = env
    b = Batch(env, [170, 99], new, 2, 4, 128, 16, 31)

    def attend(cache):
        out = q4.q4_cache_attend(b.dev[0], cache, *b.dev[2:], q_offsets=b.offsets_dev, max_q=b.max_q, return_lse=with_lse)
        return out[0] if with_lse else out

    planes = {n: p.copy() for n, p in b.planes.items()}
    key = 170 - max(1, new[0] // 2)
    ids, at = _rows_of(b, 0, [key])
    planes["v_scales"].view(np.uint16)[ids[0], 1, at[0], 1] = 0x7E00
    planes["v_codes"][ids[0], 1, at[0], 32:] = 0
    planes["v_zeros"][ids[0], 1, at[0], 1] = 0
    got, clean = (attend(c).float().cpu().numpy() for c in (to_cache(env, planes), b.cache))
    sees = np.zeros(b.q.shape[0], bool)
    sees[:new[0]] = 170 - new[0] + np.arange(new[0]) >= key
    assert sees.any() and np.isnan(got[sees][:, 4:, 64:]).all()
    keep = np.ones(got.shape, bool)
    keep[np.ix_(sees, range(4, 8), range(64, 128))] = False
    assert np.array_equal(got[keep], clean[keep])
