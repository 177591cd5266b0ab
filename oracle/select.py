"""Selection of Top-k tokens by index scores, written out as its definition --
TEST INFRASTRUCTURE ONLY (include/skv.h, skv_select).

For one unit: index keys K [n][dim], query heads q [H][dim], weights w [H], T
tokens, one key for `block` of them:

    score_j = sum_h w_h max(0, q_h . K_j)          (no max without relu)

taken: the first and last blocks asked for, then by score (a NaN below all,
the lower index first among equals), k / block in all; their tokens ascending,
-1 behind the last.

Parity status: pinned in tests/test_oracle_select.py by hand-made cases and an
enumeration of all subsets.
"""
from __future__ import annotations

import numpy as np


def scores(K: np.ndarray, q: np.ndarray, w: np.ndarray, relu: bool) -> np.ndarray:
    """float64 scores of the keys; a NaN product counts as 0 under the max."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.asarray(q, np.float64) @ np.asarray(K, np.float64).T
        if relu:
            x = np.where(x > 0, x, 0.0)
        return np.asarray(w, np.float64) @ x


def take(score: np.ndarray, T: int, k: int, block: int, first: int, last: int) -> np.ndarray:
    """The Top-k row [k] (int32) for the scores of the ceil(T / block) keys."""
    n = -(-T // block)
    s = np.array(score[:n], np.float64)
    s[np.isnan(s)] = -np.inf
    rank = [(not (j < first or j >= n - last), bool(np.isnan(score[j])), -s[j], j) for j in range(n)]
    blocks = sorted(j for *_, j in sorted(rank)[:k // block])
    tokens = [t for j in blocks for t in range(j * block, min(T, (j + 1) * block))]
    return np.array(tokens + [-1] * (k - len(tokens)), np.int32)


def select(K, q, w, T, k, block=1, first=0, last=0, relu=True) -> np.ndarray:
    n = -(-T // block)
    return take(scores(np.asarray(K)[:n], q, w, relu), T, k, block, first, last)


def on_grid(rng, shape, top: int = 32):
    """Values k / 8, |k| <= top: sums of their products are exact in fp32 in any order while they stay below 2^24 / 64."""
    return np.clip(np.rint(rng.standard_normal(shape) * 8), -top, top) / 8
