"""The selection among scores that are neighbours in fp32.

Scores are made exactly: head 0 gives 1, head 1 a whole number c <= 256 under
the weight 2^-23, so the score is 1 + c * 2^-23, the c-th fp32 number above 1.  (Both products
and their sum are exact, so the selection has to equal the definition entry for
entry.)  The rows lie in a larger buffer whose rest has to stay as it was."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Config, Context, Index

GUARD = 4096


def _want(c, nb):
    """Indices of the nb largest, the lower index first among equals, ascending."""
    return np.sort(np.lexsort((np.arange(c.size), -c))[:nb])


def _run(c, k, block=1, T_max=None, sign=1.0):
    """c [units][n] whole numbers in [0, 256]; scores sign * (1 + c * 2^-23)."""
    B, n = c.shape
    T_max = T_max or n * block
    keys = torch.zeros((B, 1, -(-T_max // block), 64), dtype=torch.bfloat16, device="cuda")
    keys[:, 0, :n, 0] = 1.0
    keys[:, 0, :n, 1] = torch.from_numpy(c.astype(np.float32)).cuda().bfloat16()
    q = torch.zeros((B, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0, 0] = q[:, :, 1, 1] = 1.0
    w = (sign * torch.tensor([1.0, 2.0 ** -23], device="cuda")).expand(B, 1, 2).contiguous()
    with Context(Config(max_requests=B, num_layers=1, max_context=T_max, topk=k, hot_slots=k, max_batch=B, row_bytes=16)) as ctx:
        req = torch.tensor([ctx.publish(n * block) for _ in range(B)], dtype=torch.int32, device="cuda")
        ix = Index(keys, block=block)
        buf = torch.full((B * k + GUARD,), -7, dtype=torch.int32, device="cuda")
        work = torch.full((ctx.select_workspace(ix, B),), 0xFF, dtype=torch.uint8, device="cuda")
        ctx.select(ix, req, q, w, buf[:B * k].view(B, 1, k), work)
        assert ctx.get_device_error() == 0
        assert bool((buf[B * k:] == -7).all()), "entries behind the last row were written"
        return buf[:B * k].view(B, k).cpu().numpy()


def _check(rows, k, block=1, **kw):
    rows = np.stack(rows)
    for i, (c, got) in enumerate(zip(rows, _run(rows, k, block, **kw))):
        if kw.get("sign") == -1.0:
            c = -c
        b = _want(c, k // block)
        assert np.array_equal(got, (b[:, None] * block + np.arange(block)).ravel()), i


def _filled(n, nb, rng, step=1, at=None):
    """Exactly nb keys of one score, key 0 `step` fp32 numbers below it, the others lower."""
    c = rng.integers(0, 2, n)
    c[rng.permutation(np.arange(1, n))[:nb] if at is None else at] = 1 + step
    c[0] = 1
    return c


# contexts of one CTA, of teams that keep their scores, of teams that read them again
SIZES = [(300, None), (3000, None), (20480, None), (40000, None), (170000, None), (400000, None), (3000, 400000)]


@pytest.mark.parametrize("block,k", [(1, 64), (1, 1000), (4, 256)])
@pytest.mark.parametrize("n,T_max", SIZES)
def test_key_0_just_below_scores_that_fill_the_selection(n, T_max, block, k):
    _fill_and_check(n, T_max, block, k)


@pytest.mark.parametrize("n", [300, 3000, 20480])
def test_key_0_just_below_in_blocks_of_64_tokens(n):
    _fill_and_check(n, None, 64, 128)


def _fill_and_check(n, T_max, block, k):
    nb = min(k // block, n - 1)
    k = nb * block
    rng = np.random.default_rng(n + k)
    rows = [_filled(n, nb, rng), _filled(n, nb, rng, step=2), _filled(n, nb, rng, at=np.arange(n - nb, n)),
            _filled(n, nb, rng, at=np.arange(1, nb + 1))]
    _check(rows, k, block, T_max=None if T_max is None else T_max * block)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n", [300, 3000, 40000, 170000])
def test_neighbouring_scores(n, sign):
    rng = np.random.default_rng(n)
    spread = [rng.integers(0, m, n) for m in (2, 3, 5, 30, 257)]
    equal = np.full(n, 9)
    equal[0] = 8  # key 0 next below more equal scores than are taken
    _check(spread + [equal], 200, sign=sign)
