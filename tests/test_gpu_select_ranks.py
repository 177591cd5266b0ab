"""The selection's ranking on score patterns where it can go wrong: many equal
scores, scores hidden from a sample, thresholds at the ends of the range, and
contexts past every size at which the kernel changes its way (scores in shared
memory or read again, one CTA or a team, one window of bits or several).

Scores are made exactly: two of a key's values hold a score's high and low
part, the query is (256, 1, 0, ...), so score = 256 a + b with |a|, |b| <= 256 is
exact in fp32."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Config, Context, Index


def _want(score, nb):
    """Indices of the nb largest, the lower index first among equals, ascending."""
    return np.sort(np.lexsort((np.arange(score.size), -score))[:nb])


def _run(scores, k, T_max=None, block=1, first=0, last=0):
    """scores: [units][n] integers in (-65536, 65536)."""
    B, n = scores.shape
    T_max = T_max or n * block
    a = np.rint(scores / 256).astype(np.float32)
    keys = torch.zeros((B, 1, -(-T_max // block), 64), dtype=torch.bfloat16, device="cuda")
    keys[:, 0, :n, 0] = torch.from_numpy(a).cuda().bfloat16()
    keys[:, 0, :n, 1] = torch.from_numpy((scores - 256 * a).astype(np.float32)).cuda().bfloat16()
    q = torch.zeros((B, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 256.0
    q[..., 1] = 1.0
    w = torch.ones((B, 1, 1), device="cuda")
    with Context(Config(max_requests=B, num_layers=1, max_context=T_max, topk=k, hot_slots=k, max_batch=B, row_bytes=16)) as ctx:
        req = torch.tensor([ctx.publish(n * block) for _ in range(B)], dtype=torch.int32, device="cuda")
        ix = Index(keys, block=block, first=first, last=last, relu=False)
        out = torch.full((B, 1, k), -7, dtype=torch.int32, device="cuda")
        work = torch.full((ctx.select_workspace(ix, B),), 0xFF, dtype=torch.uint8, device="cuda")
        ctx.select(ix, req, q, w, out, work)
        assert ctx.get_device_error() == 0
        return out.cpu().numpy()[:, 0]


SIZES = [(3000, None), (16384, None), (20480, None), (20609, None), (40000, None), (170000, None), (400000, None),
         (3000, 400000), (21000, 400000)]


def _patterns(n, k, rng):
    step = max(1, n // 2048)
    yield "distinct", rng.permutation(n) % 131000 - 65500
    yield "all equal", np.full(n, 7)
    yield "two values", np.where(rng.random(n) < 0.5, 3, 4)
    yield "few values", rng.integers(-20, 20, n)
    yield "few above many equal", np.where(np.arange(n) % max(1, n // (k // 2)) == 1, 500, -3)
    yield "ascending", np.arange(n) // 8
    yield "descending", -(np.arange(n) // 8)
    yield "one far above", np.where(np.arange(n) == n // 3, 65000, rng.integers(-9, 9, n))
    yield "the largest last", np.where(np.arange(n) >= n - k, 40000 + np.arange(n) % 1000, rng.integers(0, 30000, n))
    # what a sample of evenly spaced scores does not see, at several spacings
    for s in {step, max(1, n // 16384), 128, 64}:
        yield f"hidden from every {s}th", np.where(np.arange(n) % s == s // 2, 30000 + rng.integers(0, 9000, n), rng.integers(0, 9000, n))
    yield "narrow", 60000 + rng.integers(0, 3, n)
    yield "wide", np.sign(rng.standard_normal(n)) * np.floor(np.exp2(rng.uniform(0, 15.9, n)))


@pytest.mark.parametrize("k", [2, 100, 2048])
@pytest.mark.parametrize("n,T_max", SIZES)
def test_patterns(n, T_max, k):
    rng = np.random.default_rng(n + k)
    names, rows = zip(*_patterns(n, k, rng))
    rows = np.stack(rows).astype(np.int64)
    if n > 100000:  # a few units at a time, so that clusters share a unit
        got = np.concatenate([_run(rows[i:i + 4], k, T_max) for i in range(0, len(rows), 4)])
    else:
        got = _run(rows, k, T_max)
    for name, row, g in zip(names, rows, got):
        assert np.array_equal(g, _want(row, k)), name


@pytest.mark.parametrize("n", [20480, 400000])
def test_blocks_and_forced_blocks_of_long_contexts(n):
    rng = np.random.default_rng(n)
    rows = rng.integers(-1000, 1000, (3, n))
    got = _run(rows, 2048, block=2, first=3, last=5)
    for row, g in zip(rows, got):
        s = row.astype(float)
        s[:3] = s[n - 5:] = np.inf
        b = _want(s, 1024)
        assert np.array_equal(g, (2 * b[:, None] + np.arange(2)).ravel())


def test_more_than_a_window_of_bits():
    """Over 4 Mi keys a unit: the bits of a CTA's scores are written a window at a time."""
    n = 4_500_000
    rng = np.random.default_rng(1)
    rows = np.stack([rng.integers(-60000, 60000, n), rng.integers(0, 4, n)])
    for row, g in zip(rows, _run(rows, 2048)):
        assert np.array_equal(g, _want(row, 2048))


def test_many_entries():
    """More batch entries than score_kernel has threads, few requests, ragged."""
    rng = np.random.default_rng(2)
    R, B, k, T = 5, 700, 16, 300
    lens = [300, 0, 129, 1, 64]
    score = rng.integers(-500, 500, (R, T))
    keys = torch.zeros((R, 1, T, 64), dtype=torch.bfloat16, device="cuda")
    keys[:, 0, :, 1] = torch.from_numpy((score // 4).astype(np.float32)).cuda().bfloat16()
    ids = rng.integers(0, R, B)
    q = torch.ones((B, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    sign = np.where(rng.random(B) < 0.5, -1.0, 1.0)
    w = torch.from_numpy(sign).float().cuda().view(B, 1, 1)
    with Context(Config(max_requests=R, num_layers=1, max_context=T, topk=k, hot_slots=k, max_batch=B, row_bytes=16)) as ctx:
        for t in lens:
            ctx.publish(t)
        ix = Index(keys, relu=False)
        out = torch.full((B, 1, k), -7, dtype=torch.int32, device="cuda")
        work = torch.empty(ctx.select_workspace(ix, B), dtype=torch.uint8, device="cuda")
        ctx.select(ix, torch.from_numpy(ids).int().cuda(), q, w, out, work)
        assert ctx.get_device_error() == 0
    out = out.cpu().numpy()[:, 0]
    for b in range(B):
        t = lens[ids[b]]
        want = np.full(k, -1)
        best = _want(sign[b] * (score[ids[b], :t] // 4), k)
        want[:best.size] = best
        assert np.array_equal(out[b], want), b
