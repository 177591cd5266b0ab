"""The calls around a shared prefix as a program makes them: back to back, on several
streams, in graphs, under an SM budget, over long prefixes, with waits that run out."""
import math

import pytest
import torch

from oracle import prefix as pre
from test_gpu_prefix import SCALE, Case, _rows, context, evict

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Prefix, skv


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Step:
    """attend, weigh and evict of one batch, each reading what the call before wrote into buffers that are used again."""

    def __init__(self, B, L, n, heads, keep, seed):
        self.c = Case(B, L, n, heads, seed=seed)
        c, ctx = self.c, self.c.ctx
        self.small = Prefix(torch.zeros((L, keep, 576), device="cuda", dtype=torch.bfloat16))
        self.q = torch.empty_like(c.q)
        self.out, self.lse = torch.zeros_like(c.out[:-1]), torch.zeros_like(c.lse[:-1])
        self.out2, self.lse2 = torch.zeros_like(self.out), torch.zeros_like(self.lse)
        self.weights, self.kept = torch.zeros((L, n), device="cuda"), torch.zeros((L, keep), dtype=torch.int32, device="cuda")
        self.work = [_bytes(ctx.attend_prefix_workspace(c.prefix, B, heads)), _bytes(ctx.weigh_prefix_workspace(c.prefix, B, heads)),
                     _bytes(ctx.evict_prefix_workspace(c.prefix)), _bytes(ctx.attend_prefix_workspace(self.small, B, heads))]

    def run(self, sign):
        c, ctx = self.c, self.c.ctx
        torch.mul(c.q, sign, out=self.q)
        ctx.attend_prefix(c.prefix, self.q, self.out, self.lse, self.work[0], sm_scale=SCALE)
        ctx.weigh_prefix(c.prefix, self.q, self.lse, None, self.weights, self.work[1], sm_scale=SCALE)
        ctx.evict_prefix(c.prefix, self.weights, self.kept, self.small.rows, None, self.work[2], first=1, last=2)
        ctx.attend_prefix(self.small, self.q, self.out2, self.lse2, self.work[3], sm_scale=SCALE)
        ctx.join([self.out, self.out2], [self.lse, self.lse2], self.out, self.lse)

    def results(self):
        return [t.clone() for t in (self.out, self.lse, self.out2, self.lse2, self.weights, self.kept, self.small.rows)]


SHAPES = [(2, 1, 300, 128, 64), (5, 2, 5003, 16, 700), (40, 1, 40000, 8, 9000)]


@pytest.mark.parametrize("B,L,n,heads,keep", SHAPES)
def test_calls_without_a_pause_give_what_calls_with_one_give(B, L, n, heads, keep):
    s = Step(B, L, n, heads, keep, seed=3)
    want = []
    for sign in (1.0, -1.0):
        c = s.c.ctx
        for part in range(2):  # the second time with the device idle between the steps
            s.run(sign)
            torch.cuda.synchronize()
        want.append(s.results())
        assert c.get_device_error() == 0
    got = []
    for i in range(8):
        s.run(1.0 if i % 2 == 0 else -1.0)
        got.append(s.results())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g, want[i % 2]):
            assert torch.equal(a, b), i
    assert s.c.ctx.get_device_error() == 0


def test_two_steps_on_two_streams_and_in_two_graphs():
    """Each has a workspace of its own; the calls may overlap."""
    steps = [Step(*SHAPES[0], seed=5), Step(*SHAPES[1], seed=6), Step(*SHAPES[0], seed=7)]
    want = []
    for s in steps:
        s.run(1.0)
        torch.cuda.synchronize()
        want.append(s.results())
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run(1.0)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
    graphs = []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run(1.0)
        for t in (s.out, s.weights, s.kept, s.small.rows):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
        assert s.c.ctx.get_device_error() == 0
    del graphs


@pytest.mark.parametrize("sms", [1, 4, 10, 72, 1000])
@pytest.mark.parametrize("B,n", [(1, 700), (9, 1300)])
def test_attention_within_an_sm_budget(B, n, sms):
    c = Case(B, 2, n, seed=sms)
    c.ctx.set_attend_sms(sms)
    c.attend()
    c.check()
    c.ctx.set_attend_sms(0)
    c.attend()
    c.check()


def test_a_workspace_for_another_sm_budget_is_refused_where_it_is_too_small():
    c = Case(37, 1, 3000)
    need = {}
    for sms in (0, 4, 8, 100):
        c.ctx.set_attend_sms(sms)
        need[sms] = c.ctx.attend_prefix_workspace(c.prefix, 37)
    small, large = min(need, key=need.get), max(need, key=need.get)
    assert need[small] < need[large]
    c.ctx.set_attend_sms(large)
    with pytest.raises(skv.SkvError):
        c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, _bytes(need[small]), sm_scale=SCALE)
    work = _bytes(need[large] + 4096)
    work[need[large]:] = 99
    c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, work[:need[large]], sm_scale=SCALE)
    c.check()
    assert bool((work[need[large]:] == 99).all())  # nothing is written behind it


@pytest.mark.parametrize("B,L,n,heads", [(3, 2, 4000, 128), (9, 1, 70000, 40)])
def test_nothing_is_written_behind_a_workspace(B, L, n, heads):
    c = Case(B, L, n, heads)
    lse, w, out = c.shares(), torch.rand((L, n), device="cuda"), torch.empty((L, n), device="cuda")
    sizes = [c.ctx.attend_prefix_workspace(c.prefix, B, heads), c.ctx.weigh_prefix_workspace(c.prefix, B, heads),
             c.ctx.evict_prefix_workspace(c.prefix)]
    works = [torch.full((b + 4096,), 99, dtype=torch.uint8, device="cuda") for b in sizes]
    kept = torch.empty((L, n // 3), dtype=torch.int32, device="cuda")
    c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, works[0][:sizes[0]], sm_scale=SCALE)
    c.ctx.weigh_prefix(c.prefix, c.q, lse, w, out, works[1][:sizes[1]], sm_scale=SCALE)
    c.ctx.evict_prefix(c.prefix, w, kept, None, None, works[2][:sizes[2]])
    for b, t in zip(sizes, works):
        assert bool((t[b:] == 99).all())
    assert c.ctx.get_device_error() == 0


def test_join_without_lse():
    outs = [torch.randn((70, 512), device="cuda").bfloat16() for _ in range(3)]
    lses = [torch.randn(70, device="cuda") for _ in range(3)]
    a, b, lse = torch.empty_like(outs[0]), torch.empty_like(outs[0]), torch.empty_like(lses[0])
    with context() as ctx:
        ctx.join(outs, lses, a, lse)
        ctx.join(outs, lses, b)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        ctx.join(outs, lses, outs[0], lses[2])  # in two parts' places
        assert torch.equal(a.view(torch.int16), outs[0].view(torch.int16)) and torch.equal(lse, lses[2])


def test_queries_that_lie_off_a_border_of_16_bytes_are_refused():
    c = Case(2, 1, 300)
    flat = torch.zeros(2 * 128 * 576 + 16, device="cuda", dtype=torch.bfloat16)
    for off in (1, 2, 4):
        with pytest.raises(skv.SkvError):
            c.ctx.attend_prefix(c.prefix, flat[off:off + 2 * 128 * 576].view(2, 128, 576), c.out, c.lse, _bytes(1 << 24))
    q = c.q
    for off in (8, 16):
        c.q = flat[off:off + 2 * 128 * 576].view(2, 128, 576).copy_(q)
        c.attend()
        c.check()


def test_an_empty_batch():
    c = Case(2, 1, 300)
    none, w, out = c.q[:0], torch.rand((1, 300), device="cuda"), torch.full((1, 310), 5.0, device="cuda")
    work = _bytes(16)
    c.ctx.attend_prefix(c.prefix, none, c.out, c.lse, work, sm_scale=SCALE)
    assert bool((c.out == 7).all()) and bool((c.lse == 7).all())  # nothing is enqueued
    c.ctx.weigh_prefix(c.prefix, none, c.lse[:0], w, out, work, sm_scale=SCALE)
    assert torch.equal(out[:, :300], w) and bool((out[:, 300:] == 5).all())
    c.ctx.weigh_prefix(c.prefix, none, c.lse[:0], None, out, work, sm_scale=SCALE)
    assert not out[:, :300].any() and bool((out[:, 300:] == 5).all())


def test_a_prefix_whose_rows_lie_beyond_four_gigabytes():
    """3.9 million rows of 1152 bytes; the first and the last ones count."""
    n, heads = 3_900_001, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((1, n, 576), generator=g, device="cuda", dtype=torch.bfloat16)
    rows[:, 1000:n - 1000] *= 0.1
    q = torch.randn((1, heads, 576), generator=g, device="cuda").bfloat16()
    out, lse = torch.empty((1, heads, 512), device="cuda").bfloat16(), torch.empty((1, heads), device="cuda")
    with context() as ctx:
        p = Prefix(rows)
        w = torch.empty((1, n), device="cuda")
        ctx.attend_prefix(p, q, out, lse, _bytes(ctx.attend_prefix_workspace(p, 1, heads)), sm_scale=0.2)
        ctx.weigh_prefix(p, q, lse, None, w, _bytes(ctx.weigh_prefix_workspace(p, 1, heads)), sm_scale=0.2)
        kept, small, kw = evict(ctx, rows, w, 1200, 5, 7)
        assert ctx.get_device_error() == 0
    s = torch.cat([pre.scores(q[0], rows[0, a:a + 500_000], 0.2) for a in range(0, n, 500_000)], -1)
    want = torch.logsumexp(s, -1)
    share = torch.exp(s - want[:, None])
    o = sum(share[:, a:a + 500_000] @ rows[0, a:a + 500_000, :512].double() for a in range(0, n, 500_000))
    ds = pre.STEPS * 0.2 * float(q.abs().double().sum(-1).max()) * float(rows.abs().max())
    assert bool(((lse[0].double() - want).abs() <= ds + pre.MISC + n * 2.0 ** -24).all())
    size = sum(share[:, a:a + 500_000] @ rows[0, a:a + 500_000, :512].double().abs() for a in range(0, n, 500_000)) + o.abs()
    assert bool(((out[0].double() - o).abs() <= (pre.U_BF16 + 2 * ds + pre.MISC) * size + pre.U_BF16 * o.abs()).all())
    total = share.sum(0)
    assert bool(((w[0].double() - total).abs() <= (ds + 1e-4) * total + 1e-12).all())
    best = w[0].clone()
    best[:5] = best[n - 7:] = math.inf
    at = torch.topk(best, 1200)[1].sort()[0]
    assert torch.equal(kept[0].long(), at) and torch.equal(small[0], rows[0][at]) and torch.equal(kw[0], w[0][at])


@pytest.mark.parametrize("n,keep", [(32768, 30000), (32769, 1), (8192 * 5, 8192 * 4), (8192 * 5 + 1, 16), (4096 * 9 - 1, 5000), (300000, 299999)])
def test_eviction_at_the_borders_of_its_kernels(n, keep):
    rows, w = _rows(2, n, 0), torch.randn((2, n), device="cuda").exp()
    with context(L=2) as ctx:
        kept, out, kw = evict(ctx, rows, w, keep, min(keep, 3), 0)
    for l in range(2):
        best = w[l].clone()
        best[:min(keep, 3)] = math.inf
        at = torch.sort(best, descending=True, stable=True)[1][:keep].sort()[0]
        assert torch.equal(kept[l].long(), at) and torch.equal(out[l], rows[l][at]) and torch.equal(kw[l], w[l][at])


@pytest.mark.parametrize("kind", ["equal", "nan", "two", "forced"])
def test_eviction_of_hard_weights_from_long_prefixes(kind):
    n, keep, first, last = 100001, 30000, 7, 11
    w = torch.rand((1, n), device="cuda")
    if kind == "equal":
        w[:] = 2.0
    elif kind == "nan":
        w[w < 0.8] = math.nan
    elif kind == "two":
        w = (w > 0.9).float() - 0.5
    else:
        first, last = 10000, 20000
    rows = _rows(1, n, 0)
    with context() as ctx:
        kept, out, kw = evict(ctx, rows, w, keep, first, last)
    best = torch.where(torch.isnan(w[0]), -math.inf, w[0])
    best[:first] = best[n - last:] = math.inf
    at = torch.sort(best, descending=True, stable=True)[1][:keep].sort()[0]
    assert torch.equal(kept[0].long(), at) and torch.equal(out[0], rows[0][at])


@pytest.mark.parametrize("B,n,heads", [(2, 700, 128), (40, 9000, 16)])
def test_waits_that_run_out_end_in_an_error_bit(B, n, heads):
    """No load is issued, so nothing is in flight; the context stays usable."""
    c = Case(B, 2, n, heads, seed=8)
    work = _bytes(max(c.ctx.attend_prefix_workspace(c.prefix, B, heads), c.ctx.weigh_prefix_workspace(c.prefix, B, heads)))
    w = torch.zeros((2, n), device="cuda")
    lse = c.lse[:-1].clone()
    for out, weights in ((c.out, None), (None, w)):
        c.ctx.selftest_prefix_timeout(c.prefix, c.q, lse, out, weights, work)
        torch.cuda.synchronize()
        assert c.ctx.get_device_error() == skv.SKV_DEVERR_TIMEOUT
        assert c.ctx.get_device_error() == 0  # read and cleared
    c.out.fill_(7)
    c.attend()
    c.check()
