"""skv_select and the sticky error word: contexts of teams (clusters that share a
unit's scores), and calls that overlap one that sets the word."""
import pytest
import torch

import oracle as orc
from test_gpu_select import Case

pytestmark = pytest.mark.gpu

# one CTA a unit; teams that keep their scores; teams that read them again
CONTEXTS = [900, 40000, 400000]


@pytest.mark.parametrize("ctx", CONTEXTS)
@pytest.mark.parametrize("short", [False, True])
def test_bad_requests_and_a_set_word_fill_every_row_with_minus_one(ctx, short):
    """short: requests of fewer tokens than k (their rows need no scores)."""
    lens = [50, 64, 0] if short else [ctx, ctx - 1, 70]
    c = Case(3, 1, lens, 64, 8, 64, seed=ctx, T_max=ctx, R=4)
    good = c.req_dev
    for bad in (-1, 4):
        for at in range(3):
            ids = list(c.req)
            ids[at] = bad
            c.req_dev = torch.tensor(ids, dtype=torch.int32, device="cuda")
            c.work.fill_(0xFF)
            assert bool((c.run() == -1).all())
            c.req_dev = good
            c.work.fill_(0xFF)
            assert bool((c.run() == -1).all())  # the word is sticky
            assert c.ctx.get_device_error() == orc.E_BAD_REQUEST
    c.check(c.run())


@pytest.mark.parametrize("ctx", CONTEXTS)
def test_calls_that_overlap_one_that_sets_the_word(ctx):
    """Two selections of one context on two streams with a workspace each, one of them with a bad id: each row of the
    good one is the definition's or -1 throughout."""
    B = 4
    c = Case(B, 1, [ctx - 3 * b for b in range(B)], 64, 8, 64, seed=ctx + 1, R=B + 1)
    want = torch.stack([torch.from_numpy(c.want(b, 0)) for b in range(B)]).cuda()
    other = torch.full_like(c.work, 0xFF)
    bad = c.req_dev.clone()
    bad[B - 1] = B + 1
    spare = torch.empty((B, 1, 64), dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(30):
        outs = [torch.full((B, 1, 64), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        for j, out in enumerate(outs):
            c.ctx.select(c.index, c.req_dev, c.q, c.w, out, c.work, stream=streams[0])
            if j == i % 3:
                c.ctx.select(c.index, bad, c.q, c.w, spare, other, stream=streams[1])
        torch.cuda.synchronize()
        assert bool((spare == -1).all())
        for out in outs:
            ok = (out[:, 0] == want).all(-1) | (out[:, 0] == -1).all(-1)
            assert bool(ok.all()), i
        assert c.ctx.get_device_error() == orc.E_BAD_REQUEST
        c.work.fill_(0xFF)
    c.check(c.run())
