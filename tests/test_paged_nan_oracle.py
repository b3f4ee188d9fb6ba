"""The oracle's attention of queries that are not finite: NaN, but for a row that sees no key."""
import numpy as np
import pytest

from oracle import paged as ref


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf], ids=str)
def test_a_query_that_is_not_finite(bad):
    rng = np.random.default_rng(1)
    kp, vp = rng.standard_normal((2, 1, 3, 4, 1, 8)).astype(np.float32)
    q = rng.standard_normal((1, 5, 2, 8)).astype(np.float32)
    clean, _, _ = ref.paged_attention(q, kp, vp, [[2, 0, 1]], [0, 5], [3])
    q[0, 1, 0, 2] = q[0, 4, 1, 0] = bad
    out, lse, _ = ref.paged_attention(q, kp, vp, [[2, 0, 1]], [0, 5], [3])
    hit = np.zeros(q.shape[:-1], bool)
    hit[0, 1, 0] = hit[0, 4, 1] = True
    assert np.all(np.isnan(out[hit])) and np.array_equal(out[~hit], clean[~hit]) and not np.any(np.isfinite(lse[hit]))


def test_only_scores_of_minus_infinity():
    k = np.ones((1, 1, 4, 1, 2), np.float32)
    out, lse, _ = ref.paged_attention(np.array([[[[-np.inf, 1.0]]]], np.float32), k, k, [[0]], [0, 1], [0])
    assert np.all(np.isnan(out)) and np.all(np.isneginf(lse))


def test_a_row_that_sees_nothing_is_zeros_whatever_its_query_holds():
    k = np.ones((1, 1, 4, 1, 2), np.float32)
    t = np.ones((1, 1, 2, 1, 2), np.float32)
    q = np.full((1, 1, 2, 1, 2), np.nan, np.float32)
    out, lse, _ = ref.paged_tree_attention(q, k, k, [[0]], t, t, np.array([[0], [1]], np.int32), [0])
    assert np.all(out[0, 0, 0] == 0) and np.isneginf(lse[0, 0, 0, 0]) and np.all(np.isnan(out[0, 0, 1]))
