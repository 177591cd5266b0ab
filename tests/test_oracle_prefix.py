"""The shared prefix's oracle against hand-made cases and identities (CPU only)."""
import itertools
import math

import pytest
import torch

from oracle import prefix as pre


def _case(i, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((i, 576), generator=g, dtype=torch.float64), torch.randn((n, 576), generator=g, dtype=torch.float64)


def test_by_hand():
    q, rows = torch.zeros((2, 576)), torch.zeros((3, 576))
    q[0, 0], q[1, 575] = 1.0, 2.0
    rows[0, 0], rows[1, 575], rows[2, 1] = math.log(2), math.log(3), 7.0
    out, lse, *_ = pre.attend(q, rows, 1.0)
    assert torch.allclose(lse.exp(), torch.tensor([4.0, 11.0], dtype=torch.float64))  # 2 + 1 + 1, 1 + 9 + 1
    assert torch.allclose(out[0, :2], torch.tensor([math.log(2) / 2, 7 / 4], dtype=torch.float64))
    assert torch.allclose(out[1, :2], torch.tensor([math.log(2) / 11, 7 / 11], dtype=torch.float64))
    w, _ = pre.weigh(q, rows, lse, 1.0, before=torch.tensor([1.0, 0, 0]), gain=2.0)
    assert torch.allclose(w, torch.tensor([1 + 2 * (2 / 4 + 1 / 11), 2 * (1 / 4 + 9 / 11), 2 * (1 / 4 + 1 / 11)], dtype=torch.float64))


def test_an_empty_prefix():
    out, lse, *_ = pre.attend(torch.ones((4, 576)), torch.ones((0, 576)), 1.0)
    assert not out.any() and bool((lse == -math.inf).all())
    w, _ = pre.weigh(torch.ones((2, 576)), torch.ones((3, 576)), torch.tensor([-math.inf, -math.inf]), 1.0)
    assert not w.any()


@pytest.mark.parametrize("cut", [1, 17, 40])
def test_a_split_prefix_joined_is_the_whole(cut):
    q, rows = _case(5, 41)
    out, lse, *_ = pre.attend(q, rows, 0.05)
    a, b = pre.attend(q, rows[:cut], 0.05), pre.attend(q, rows[cut:], 0.05)
    o, e = pre.join([a[0], b[0], torch.full_like(out, math.nan)], [a[1], b[1], torch.full_like(lse, -math.inf)])
    assert torch.allclose(o, out, rtol=1e-12, atol=1e-14) and torch.allclose(e, lse, rtol=1e-13)


def test_shares_sum_to_the_heads():
    q, rows = _case(6, 30, seed=1)
    lse = pre.attend(q, rows, 0.1)[1]
    w, _ = pre.weigh(q, rows, lse, 0.1)
    assert abs(float(w.sum()) - 6) < 1e-12


@pytest.mark.parametrize("seed", range(4))
def test_no_other_tokens_weigh_more(seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-2, 3, (8,), generator=g).double()
    for keep, first, last in ((1, 0, 0), (4, 1, 1), (5, 0, 3), (8, 0, 0), (9, 2, 2)):
        got = pre.evict(w, keep, first, last)
        forced = {j for j in range(8) if j < first or j >= 8 - last}
        assert forced <= set(got) and got == sorted(got) and len(got) == min(keep, 8)
        best = max(float(sum(w[j] for j in c)) for c in itertools.combinations(range(8), len(got)) if forced <= set(c))
        assert sum(float(w[j]) for j in got) == best
        free = [j for j in got if j not in forced]
        for j in free:  # ties to the lower index
            assert all(i in got for i in range(j) if w[i] >= w[j])


def test_a_nan_is_the_lightest():
    w = torch.tensor([math.nan, -math.inf, 1.0, math.nan, math.inf])
    assert pre.evict(w, 3, 0, 0) == [1, 2, 4] and pre.evict(w, 4, 0, 0) == [0, 1, 2, 4]
