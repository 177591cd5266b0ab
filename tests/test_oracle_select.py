"""The selection's oracle against hand-made rows and an enumeration of all
subsets (CPU only)."""
import itertools

import numpy as np
import pytest

from oracle import select as sel


def test_by_hand():
    K = np.array([[1.0, 0], [2, 0], [0, 5], [-3, 1], [2, 0], [0, 0]])
    q = np.array([[1.0, 0], [0, 1]])
    w = np.array([1.0, 0.25])
    assert list(sel.scores(K, q, w, True)) == [1, 2, 1.25, 0.25, 2, 0]
    assert list(sel.scores(K, q, w, False)) == [1, 2, 1.25, -2.75, 2, 0]
    assert list(sel.select(K, q, w, 6, 1)) == [1]          # the lower of two equals
    assert list(sel.select(K, q, w, 6, 3)) == [1, 2, 4]
    assert list(sel.select(K, q, w, 4, 3)) == [0, 1, 2]    # keys behind the length do not count
    assert list(sel.select(K, q, w, 2, 3)) == [0, 1, -1]
    assert list(sel.select(K, q, w, 0, 3)) == [-1, -1, -1]
    assert list(sel.select(K, q, w, 6, 3, first=1, last=1)) == [0, 1, 5]
    assert list(sel.select(K, q, w, 11, 4, block=2)) == [2, 3, 8, 9]
    assert list(sel.select(K, q, w, 11, 4, block=2, last=1)) == [2, 3, 10, -1]  # the last block is cut short


def test_nan_and_infinite_scores():
    K = np.array([[np.nan], [1.0], [np.inf], [-1.0]])
    q, w = np.array([[1.0]]), np.array([1.0])
    assert list(sel.select(K, q, w, 4, 2)) == [1, 2]
    assert list(sel.select(K, q, w, 4, 3)) == [0, 1, 2]            # under the max a NaN is 0, as -1 is
    assert list(sel.select(K, q, w, 4, 3, relu=False)) == [1, 2, 3]  # without it a NaN is below all


@pytest.mark.parametrize("seed", range(5))
def test_no_subset_is_better(seed):
    rng = np.random.default_rng(seed)
    s = rng.integers(-3, 4, 9).astype(float)
    for nb in (1, 3, 8):
        got = [t for t in sel.take(s, 9, nb, 1, 0, 0) if t >= 0]
        best = max(itertools.combinations(range(9), nb), key=lambda c: (sorted((s[j] for j in c), reverse=True), [-j for j in c]))
        assert sorted(s[j] for j in got) == sorted(s[j] for j in best)
        for j in got:  # ties to the lower index
            assert all(i in got for i in range(j) if s[i] >= s[j])
