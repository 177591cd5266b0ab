"""A prefix that a batch shares, on the GPU: attention over it, the join, the tokens'
weights and the eviction, against their definitions in 64 bits (oracle/prefix.py,
with the bounds derived there)."""
import math

import pytest
import torch

from oracle import prefix as pre

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Config, Context, Prefix, SkvError

SCALE = 1.0 / 24.0


def context(B=1, L=1, **kw):
    return Context(Config(max_requests=1, num_layers=L, max_context=1, topk=1, hot_slots=1, max_batch=B, **kw))


class Case:
    """A batch's queries and a prefix whose rows lie apart, with NaN between and behind them."""

    def __init__(self, B, L, n, heads=128, seed=0, gap=64, loud=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.L, self.n, self.heads = B, L, n, heads
        wide = torch.full((L, n + 3, 576 + gap), math.nan, device="cuda", dtype=torch.bfloat16)
        wide[:, :n, :576] = (torch.randn((L, n, 576), generator=g, device="cuda") *
                             torch.exp2(2 * torch.rand((L, n, 1), generator=g, device="cuda") - 1)).bfloat16()
        self.rows = wide[:, :n, :576]
        self.q = (loud * torch.randn((B * L, heads, 576), generator=g, device="cuda")).bfloat16()
        self.ctx = context(B, L)
        self.prefix = Prefix(self.rows)
        self.out = torch.full((B * L + 1, heads, 512), 7.0, device="cuda", dtype=torch.bfloat16)  # one unit more than is written
        self.lse = torch.full((B * L + 1, heads), 7.0, device="cuda")

    def layer(self, l, t=None):
        """The query rows of a layer (or those of t [units][heads]...), entries and heads in order."""
        t = self.q if t is None else t
        return t[:self.B * self.L].unflatten(0, (self.B, self.L))[:, l].flatten(0, 1)

    def attend(self, **kw):
        layer = kw.get("layer", -1)
        work = torch.empty(self.ctx.attend_prefix_workspace(self.prefix, self.B, self.heads, layer), dtype=torch.uint8, device="cuda")
        kw.setdefault("sm_scale", SCALE)
        self.ctx.attend_prefix(self.prefix, self.q, self.out, self.lse, work, B=self.B, **kw)
        return self.out, self.lse

    def check(self, scale=SCALE):
        for l in range(self.L):
            out, lse, out_off, lse_off = pre.attend(self.layer(l), self.rows[l], scale)
            got, got_lse = self.layer(l, self.out).double(), self.layer(l, self.lse).double()
            over = ((got - out).abs() - out_off).amax()
            assert over <= 0, (l, float(over), float((got - out).abs().amax()))
            if self.n:
                assert ((got_lse - lse).abs() <= lse_off).all(), (l, float((got_lse - lse).abs().amax()))
            else:
                assert (got_lse == lse).all()
        assert bool((self.out[-1] == 7).all()) and bool((self.lse[-1] == 7).all())  # what lies behind the last unit
        assert self.ctx.get_device_error() == 0

    def weigh(self, lse, before, out=None, **kw):
        out = torch.empty_like(before) if out is None else out
        work = torch.empty(self.ctx.weigh_prefix_workspace(self.prefix, self.B, self.heads, kw.get("layer", -1)), dtype=torch.uint8,
                           device="cuda")
        self.ctx.weigh_prefix(self.prefix, self.q, lse, before, out, work, sm_scale=SCALE, B=self.B, **kw)
        return out

    def shares(self):
        """An lse of which the prefix is about a half."""
        lse = torch.empty((self.B * self.L, self.heads), device="cuda")
        for l in range(self.L):
            lse.unflatten(0, (self.B, self.L))[:, l] = (pre.attend(self.layer(l), self.rows[l], SCALE)[1].view(self.B, self.heads) + 0.7).float()
        return lse


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4096, 5003])
@pytest.mark.parametrize("B,L", [(1, 1), (2, 1), (3, 2)])
def test_attention_over_prefixes_of_any_length(B, L, n):
    c = Case(B, L, n, seed=n)
    c.attend()
    c.check()


@pytest.mark.parametrize("heads", [1, 2, 7, 16, 37, 40, 64, 65, 127, 128])
@pytest.mark.parametrize("B,n", [(1, 70), (5, 300), (19, 130)])
def test_attention_of_any_number_of_heads(B, heads, n):
    c = Case(B, 2, n, heads, seed=heads)
    c.attend()
    c.check()


@pytest.mark.parametrize("B,L,n,heads", [(40, 2, 700, 128), (160, 1, 330, 128), (77, 3, 200, 128), (192, 4, 130, 16), (1, 8, 20000, 128)])
def test_attention_of_large_batches_and_long_prefixes(B, L, n, heads):
    c = Case(B, L, n, heads, seed=B)
    c.attend()
    c.check()


def test_attention_over_an_empty_prefix():
    c = Case(3, 2, 0)
    out, lse = c.attend()
    assert not out[:6].any() and bool((lse[:6] == -math.inf).all())
    c.check()


@pytest.mark.parametrize("loud", [1e-3, 8.0, 60.0])
def test_attention_whose_scores_hardly_differ_or_differ_widely(loud):
    c = Case(3, 1, 900, loud=loud)
    c.attend()
    c.check()


@pytest.mark.parametrize("n", [64, 200, 1500])
def test_attention_whose_maximum_keeps_rising(n):
    """Scores that rise along the prefix, by far more than a stale reference may be off."""
    c = Case(2, 1, n)
    c.q[..., 1:] = 0
    c.q[..., 0] = 8.0
    c.rows[0, :, 0] = torch.arange(n, device="cuda").bfloat16() * 0.5
    c.attend(sm_scale=1.0)
    c.check(1.0)


def test_attention_with_one_token_far_above_the_others():
    c = Case(2, 1, 777)
    c.q[..., 0] = 30.0
    c.rows[0, 700, 0] = 100.0
    c.attend(sm_scale=1.0)
    c.check(1.0)


def test_attention_on_one_layer():
    c = Case(4, 3, 210)
    whole = [t.clone() for t in c.attend()]
    c.check()
    q = c.q
    for l in range(3):
        c.q = q.view(4, 3, 128, 576)[:, l].contiguous()
        out, lse = c.attend(layer=l)
        assert torch.equal(out[:4].float(), whole[0][:-1].view(4, 3, 128, 512)[:, l].float()) or \
            torch.allclose(out[:4].float(), whole[0][:-1].view(4, 3, 128, 512)[:, l].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
        assert torch.allclose(lse[:4], whole[1][:-1].view(4, 3, 128)[:, l], rtol=1e-5)


def test_a_nan_stays_with_the_heads_it_meets():
    c = Case(2, 1, 300)
    c.q[1, 5, 9] = math.nan
    out, lse = c.attend()
    bad = torch.zeros((2, 128), dtype=torch.bool, device="cuda")
    bad[1, 5] = True
    assert bool(torch.isnan(lse[:2]).eq(bad).all()) and bool(torch.isnan(out[:2]).all(-1).eq(bad).all())
    assert not bool(torch.isnan(out[:2][~bad]).any())
    c.rows[0, 250, 570] = math.nan
    out, lse = c.attend()
    assert bool(torch.isnan(lse[:2]).all()) and bool(torch.isnan(out[:2]).all())


def test_attention_without_lse_and_twice_the_same():
    c = Case(3, 1, 5000)
    out = c.attend()[0].clone()
    lse, c.lse = c.lse, None
    c.attend()
    assert torch.equal(out.view(torch.int16), c.out.view(torch.int16))
    c.lse = lse
    c.check()


# ----------------------------------------------------------------------- join
@pytest.mark.parametrize("parts", range(1, 9))
@pytest.mark.parametrize("rows", [1, 9, 1000])
def test_join(parts, rows):
    g = torch.Generator(device="cuda").manual_seed(parts)
    outs = [torch.randn((rows, 512), generator=g, device="cuda").bfloat16() for _ in range(parts)]
    lses = [3 * torch.randn(rows, generator=g, device="cuda") for _ in range(parts)]
    for i, (o, e) in enumerate(zip(outs, lses)):
        none = torch.arange(rows, device="cuda") % (i + 2) == 0
        e[none] = -math.inf
        o[none] = math.nan  # whatever it holds
    out, lse = torch.full((rows + 1, 512), 7.0, device="cuda").bfloat16(), torch.full((rows + 1,), 7.0, device="cuda")
    with context() as ctx:
        ctx.join(outs, lses, out[:rows], lse[:rows])
        _check_join(outs, lses, out[:rows], lse[:rows])
        assert bool((out[rows:] == 7).all()) and bool((lse[rows:] == 7).all())
        ctx.join(outs, lses, outs[-1], lses[-1])  # in a part's place
        assert torch.equal(outs[-1].view(torch.int16), out[:rows].view(torch.int16)) and torch.equal(lses[-1], lse[:rows])


def _check_join(outs, lses, out, lse):
    want, want_lse = pre.join(outs, lses)
    size = pre.join([o.abs() for o in outs], lses)[0]
    # each share is off by at most 2^-20 (two exponentials' arguments of at most 2^5, a sum of 8, a division), out is rounded once
    assert bool(((out.double() - want).abs() <= pre.U_BF16 * want.abs() + 2.0 ** -18 * size + 1e-30).all())
    none = want_lse == -math.inf
    assert bool((lse.double() == want_lse)[none].all()) and not bool(out[none].any())
    assert bool(((lse.double() - want_lse).abs()[~none] <= 2.0 ** -21 * (1 + want_lse.abs()[~none])).all())


def test_join_passes_a_nan_on():
    outs = [torch.ones((3, 512), device="cuda").bfloat16() for _ in range(2)]
    lses = [torch.tensor([0.0, math.nan, 1.0], device="cuda"), torch.tensor([1.0, 0.0, -math.inf], device="cuda")]
    out, lse = torch.empty_like(outs[0]), torch.empty_like(lses[0])
    with context() as ctx:
        ctx.join(outs, lses, out, lse)
    assert bool(torch.isnan(out).all(-1).eq(torch.tensor([False, True, False], device="cuda")).all())
    assert bool(torch.isnan(lse).eq(torch.tensor([False, True, False], device="cuda")).all())


def test_a_split_prefix_joined_is_the_whole():
    c = Case(5, 1, 1300)
    whole, whole_lse = (t[:5].clone() for t in c.attend())
    parts = []
    for a, b in ((0, 0), (0, 1), (1, 700), (700, 1300)):
        c.prefix.rows = c.rows[:, a:b]
        out, lse = c.attend()
        parts.append((out[:5].clone(), lse[:5].clone()))
    c.prefix.rows = c.rows
    c.ctx.join([o for o, _ in parts], [e for _, e in parts], c.out[:5], c.lse[:5])
    assert torch.allclose(c.lse[:5], whole_lse, rtol=1e-5, atol=1e-5)
    # each part is rounded once more on the way
    out, _, off, _ = pre.attend(c.layer(0), c.rows[0], SCALE)
    size = sum((torch.exp(e.double() - whole_lse.double())[..., None] * o.double().abs().nan_to_num()) for o, e in parts).flatten(0, 1)
    assert bool(((c.layer(0, c.out).double() - out).abs() <= off + pre.U_BF16 * size).all())
    assert bool(((c.layer(0, c.out).double() - whole.flatten(0, 1).double()).abs() <= 2 * off + pre.U_BF16 * size).all())


# -------------------------------------------------------------------- weights
def _check_weights(c, got, lse, before, gain=1.0, layers=None):
    for l in range(c.L) if layers is None else layers:
        want, off = pre.weigh(c.layer(l), c.rows[l], c.layer(l, lse), SCALE, None if before is None else before[l, :c.n], gain)
        over = ((got[l, :c.n].double() - want).abs() - off).amax() if c.n else 0
        assert over <= 0, (l, float(over))
    assert c.ctx.get_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 63, 127, 128, 129, 255, 256, 257, 1000, 5003])
@pytest.mark.parametrize("B,L", [(1, 1), (2, 1), (3, 2)])
def test_weights_over_prefixes_of_any_length(B, L, n):
    c = Case(B, L, n, seed=n)
    lse, before = c.shares(), torch.rand((L, n), device="cuda")
    _check_weights(c, c.weigh(lse, before), lse, before)


@pytest.mark.parametrize("heads", [1, 2, 7, 16, 37, 40, 64, 65, 127, 128])
@pytest.mark.parametrize("B,n", [(1, 70), (5, 300), (19, 130)])
def test_weights_of_any_number_of_heads(B, heads, n):
    c = Case(B, 2, n, heads, seed=heads)
    lse, before = c.shares(), torch.rand((2, n), device="cuda")
    _check_weights(c, c.weigh(lse, before), lse, before)


@pytest.mark.parametrize("B,L,n,heads", [(40, 2, 700, 128), (160, 1, 330, 128), (77, 3, 200, 128), (192, 4, 130, 16), (1, 8, 20000, 128)])
def test_weights_of_large_batches_and_long_prefixes(B, L, n, heads):
    c = Case(B, L, n, heads, seed=B)
    lse, before = c.shares(), torch.rand((L, n), device="cuda")
    _check_weights(c, c.weigh(lse, before), lse, before)


def test_weights_in_wider_buffers_with_a_gain_and_in_place():
    c = Case(3, 2, 300)
    lse = c.shares()
    wide = torch.full((2, 350), 3.0, device="cuda")
    once = c.weigh(lse, None, out=wide, gain=2.5)
    assert bool((wide[:, 300:] == 3).all())
    _check_weights(c, once, lse, None, 2.5)
    before = wide.clone()
    c.weigh(lse, wide, out=wide, gain=-1.0)
    _check_weights(c, wide, lse, before, -1.0)
    assert bool((wide[:, 300:] == 3).all())


def test_weights_on_one_layer():
    c = Case(4, 3, 210)
    lse, before = c.shares(), torch.rand((3, 210), device="cuda")
    whole = c.weigh(lse, before)
    q = c.q
    for l in range(3):
        c.q = q.view(4, 3, 128, 576)[:, l].contiguous()
        out = torch.full_like(before, 9.0)
        c.weigh(lse.view(4, 3, 128)[:, l].contiguous(), before, out=out, layer=l)
        assert torch.allclose(out[l], whole[l], rtol=1e-5) and bool((out[[x for x in range(3) if x != l]] == 9).all())


def test_heads_that_attended_to_nothing_add_nothing():
    c = Case(3, 1, 500)
    lse, before = c.shares(), torch.zeros((1, 500), device="cuda")
    lse[1] = -math.inf
    lse[2, 7] = -math.inf
    got = c.weigh(lse, before)
    _check_weights(c, got, lse, before)
    lse[:] = -math.inf
    assert not bool(c.weigh(lse, before).any())


@pytest.mark.parametrize("B,heads", [(4, 40), (1, 128), (3, 37)])
def test_an_infinite_key_that_no_head_attends_to_weighs_nothing(B, heads):
    """Tiles that are not full, and heads that attended to nothing, meet it with zeros."""
    c = Case(B, 1, 300, heads)
    lse = c.shares()
    c.q[..., 3] = -1.0
    c.rows[0, 17, 3] = math.inf
    lse[0, 2] = -math.inf
    c.q[0, 2] = 0.0
    got = c.weigh(lse, torch.zeros((1, 300), device="cuda"))
    assert got[0, 17] == 0 and not bool(torch.isnan(got).any())


def test_weights_twice_are_the_same():
    c = Case(50, 1, 900)
    lse, before = c.shares(), torch.rand((1, 900), device="cuda")
    assert torch.equal(c.weigh(lse, before), c.weigh(lse, before))


# ------------------------------------------------------------------- eviction
def evict(ctx, rows, weights, keep, first=0, last=0, layer=-1, with_rows=True):
    p = Prefix(rows)
    layers = 1 if layer >= 0 else rows.shape[0]
    kept = torch.full((layers, keep), -7, dtype=torch.int32, device="cuda")
    out = torch.full((layers, keep, 576), 7.0, device="cuda", dtype=torch.bfloat16) if with_rows else None
    w = torch.full((layers, keep), 7.0, device="cuda") if with_rows else None
    work = torch.empty(ctx.evict_prefix_workspace(p, layer), dtype=torch.uint8, device="cuda")
    ctx.evict_prefix(p, weights, kept, out, w, work, first=first, last=last, layer=layer)
    return kept, out, w


def check_evicted(rows, weights, keep, first, last, got):
    kept, out, w = got
    for l in range(rows.shape[0]):
        n = rows.shape[1]
        want = pre.evict(weights[l, :n].tolist(), keep, first, last)
        m = len(want)
        assert kept[l, :m].tolist() == want and bool((kept[l, m:] == -1).all())
        at = torch.tensor(want, dtype=torch.long, device="cuda")
        assert torch.equal(out[l, :m].view(torch.int16), rows[l][at].view(torch.int16)) and bool((out[l, m:] == 7).all())
        assert torch.equal(w[l, :m].view(torch.int32), weights[l][at].view(torch.int32)) and bool((w[l, m:] == 7).all())


def _rows(L, n, gap=64):
    x = torch.randn((L, n, 576 + gap), device="cuda").bfloat16()
    return x[..., :576]


@pytest.mark.parametrize("n,keep,first,last", [
    (1, 1, 0, 0), (1, 5, 1, 1), (2, 1, 0, 0), (2, 1, 0, 1), (100, 33, 0, 0), (100, 100, 50, 50), (100, 101, 0, 0), (100, 99, 0, 99),
    (129, 64, 4, 8), (1000, 1, 0, 0), (1000, 10, 10, 0), (4096, 1024, 4, 64), (5003, 4999, 0, 1), (20500, 700, 1, 600),
    (70001, 20000, 3, 5), (200000, 150000, 10, 10)])
def test_eviction(n, keep, first, last):
    L = 3 if n < 10000 else 1
    torch.manual_seed(n)
    rows, weights = _rows(L, n), torch.exp(3 * torch.randn((L, n), device="cuda"))
    with context(L=L) as ctx:
        check_evicted(rows, weights, keep, first, last, evict(ctx, rows, weights, keep, first, last))
        assert ctx.get_device_error() == 0


@pytest.mark.parametrize("kind", ["equal", "two", "zero", "nan", "all nan", "inf", "neighbours", "negative"])
@pytest.mark.parametrize("n,keep", [(700, 300), (30000, 4000)])
def test_eviction_of_hard_weights(kind, n, keep):
    torch.manual_seed(n)
    w = torch.rand((2, n), device="cuda")
    at = torch.rand((2, n), device="cuda") < 0.3
    if kind == "equal":
        w[:] = 0.25
    elif kind == "two":
        w = (w > 0.95).float()
    elif kind == "zero":
        w = torch.where(at, 0.0, -0.0)
    elif kind == "nan":
        w[at] = math.nan
    elif kind == "all nan":
        w[:] = math.nan
    elif kind == "inf":
        w[at] = math.inf
        w[~at & (w < 0.3)] = -math.inf
    elif kind == "neighbours":
        w = (1.0 + (w * 8).floor() * 2.0 ** -23)
    else:
        w = -torch.exp(20 * w)
    rows = _rows(2, n)
    with context(L=2) as ctx:
        check_evicted(rows, w, keep, 3, 5, evict(ctx, rows, w, keep, 3, 5))


def test_eviction_on_one_layer_and_without_rows():
    rows, w = _rows(3, 900), torch.rand((3, 1000), device="cuda")
    with context(L=3) as ctx:
        whole = evict(ctx, rows, w, 200, 4, 9)
        check_evicted(rows, w, 200, 4, 9, whole)
        for l in range(3):
            one = evict(ctx, rows, w, 200, 4, 9, layer=l)
            assert all(torch.equal(a[0].float(), b[l].float()) for a, b in zip(one, whole))
        assert torch.equal(evict(ctx, rows, w, 200, 4, 9, with_rows=False)[0], whole[0])


def test_eviction_from_an_empty_prefix():
    with context() as ctx:
        kept, out, w = evict(ctx, _rows(1, 0), torch.empty((1, 0), device="cuda"), 5)
        assert bool((kept == -1).all()) and bool((out == 7).all()) and bool((w == 7).all())


# ---------------------------------------------------------------- as one step
def test_a_step_over_a_shared_prefix_and_its_eviction():
    """Own tokens and prefix attended and joined, the prefix weighed and cut, and attended again; eagerly and replayed."""
    B, L, T, k, n, keep = 4, 2, 500, 128, 1000, 300
    torch.manual_seed(5)
    ctx = Context(Config(max_requests=B, num_layers=L, max_context=T, topk=k, hot_slots=k, max_batch=B))
    own = torch.randn((B, L, T, 576), device="cuda").bfloat16()
    rows = torch.randn((L, n, 576), device="cuda").bfloat16()
    q = torch.randn((B * L, 128, 576), device="cuda").bfloat16()
    req = torch.tensor([ctx.publish(T, rows=own[b].contiguous().view(torch.uint8)) for b in range(B)], dtype=torch.int32, device="cuda")
    topk = torch.rand((B, L, T), device="cuda").argsort(-1)[..., :k].to(torch.int32).contiguous()
    slots, count = torch.empty_like(topk), torch.empty((2, B, L), dtype=torch.int32, device="cuda")
    prefix, small = Prefix(rows), Prefix(torch.zeros((L, keep, 576), device="cuda", dtype=torch.bfloat16))
    outs = [torch.zeros((B * L, 128, 512), device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    lses = [torch.zeros((B * L, 128), device="cuda") for _ in range(4)]
    weights, kept, kept_w = torch.zeros((L, n), device="cuda"), torch.zeros((L, keep), dtype=torch.int32, device="cuda"), torch.zeros((L, keep), device="cuda")
    work = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in (
        ctx.attend_prefix_workspace(prefix, B), ctx.weigh_prefix_workspace(prefix, B), ctx.evict_prefix_workspace(prefix))]

    def step():
        ctx.assemble(req, topk, slots, count[0], count[1])
        ctx.attend(req, q.view(torch.int16), slots, outs[0].view(torch.int16), lses[0], sm_scale=SCALE)
        ctx.attend_prefix(prefix, q, outs[1], lses[1], work[0], sm_scale=SCALE)
        ctx.join(outs[:2], lses[:2], outs[2], lses[2])
        ctx.weigh_prefix(prefix, q, lses[2], None, weights, work[1], sm_scale=SCALE)
        ctx.evict_prefix(prefix, weights, kept, small.rows, kept_w, work[2], first=4, last=16)
        ctx.attend_prefix(small, q, outs[3], lses[3], work[0], sm_scale=SCALE)

    step()
    torch.cuda.synchronize()
    assert ctx.get_device_error() == 0
    first = [t.clone() for t in (outs[2], lses[2], weights, kept, small.rows, kept_w, outs[3], lses[3])]
    for u in range(B * L):
        b, l = divmod(u, L)
        picked = torch.cat((own[b, l][topk[b, l].long()], rows[l]))
        out, lse, off, lse_off = pre.attend(q[u], picked, SCALE)
        # the parts are rounded once more than the whole; their scores cross a pair of CTAs as 24 bits (2^-16 of a score)
        slack = 2.0 ** -15 * SCALE * (q[u].double().abs() @ picked.double().abs().T).amax(-1)
        assert bool(((lses[2][u].double() - lse).abs() <= lse_off + slack).all())
        size = torch.softmax(pre.scores(q[u], picked, SCALE), -1) @ picked[:, :512].double().abs()
        assert bool(((outs[2][u].double() - out).abs() <= off + (pre.U_BF16 + 2 * slack[:, None]) * (size + out.abs())).all())
        out, lse, off, lse_off = pre.attend(q[u], small.rows[l], SCALE)
        assert bool(((outs[3][u].double() - out).abs() <= off).all()) and bool(((lses[3][u].double() - lse).abs() <= lse_off).all())
    for l in range(L):
        want, off = pre.weigh(q.view(B, L, 128, 576)[:, l].flatten(0, 1), rows[l], lses[2].view(B, L, 128)[:, l].flatten(), SCALE)
        assert bool(((weights[l].double() - want).abs() <= off).all())
        at = pre.evict(weights[l].tolist(), keep, 4, 16)
        assert kept[l].tolist() == at and torch.equal(small.rows[l], rows[l][at]) and torch.equal(kept_w[l], weights[l][at])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (outs[2], lses[2], weights, small.rows, outs[3]):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert ctx.get_device_error() == 0
    for a, b in zip(first, (outs[2], lses[2], weights, kept, small.rows, kept_w, outs[3], lses[3])):
        assert torch.equal(a, b)
    del graph
    ctx.close()


# ------------------------------------------------------------------- refusals
def test_what_is_refused():
    """Nothing of a refused call is enqueued."""
    c = Case(2, 2, 100)
    work = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    ok = dict(sm_scale=SCALE)

    def attend(prefix=c.prefix, q=c.q, out=c.out, lse=c.lse, work=work, **kw):
        c.ctx.attend_prefix(prefix, q, out, lse, work, **{**ok, **kw})

    attend()
    for bad in (dict(layer=-2), dict(layer=2), dict(B=3), dict(B=-1), dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(sm_scale=math.inf),
                dict(sm_scale=math.nan), dict(work=work[:8]), dict(work=work[1:]), dict(q=torch.empty((4, 129, 576), device="cuda").bfloat16(),
                out=torch.empty((4, 129, 512), device="cuda").bfloat16(), lse=None)):
        with pytest.raises((SkvError, ValueError)):
            attend(**bad)
    flat = torch.zeros(2 * 100 * 584 + 64, device="cuda").bfloat16()
    for rows in (flat.as_strided((2, 100, 576), (58400, 580, 1)),      # row stride no multiple of 16 bytes
                 flat.as_strided((2, 100, 576), (58404, 584, 1)),      # layer stride
                 flat.as_strided((2, 100, 576), (58400, 568, 1)),      # rows that overlap
                 flat[4:].as_strided((2, 100, 576), (58400, 584, 1))):  # not 16-byte aligned
        with pytest.raises(SkvError):
            attend(prefix=Prefix(rows))
    with pytest.raises(ValueError):
        attend(prefix=Prefix(c.rows[:1]))
    w = torch.zeros((2, 100), device="cuda")
    lse = torch.zeros((4, 128), device="cuda")
    for bad in (dict(gain=math.inf), dict(gain=math.nan), dict(sm_scale=0.0), dict(layer=5)):
        with pytest.raises(SkvError):
            c.ctx.weigh_prefix(c.prefix, c.q, lse, w, w, work, **{**ok, **bad})
    for weights in (w[:, :99], w[:1], w.double(), torch.zeros((100, 2), device="cuda").T):
        with pytest.raises(ValueError):
            c.ctx.weigh_prefix(c.prefix, c.q, lse, weights, w, work, **ok)
        with pytest.raises(ValueError):
            c.ctx.weigh_prefix(c.prefix, c.q, lse, w, weights, work, **ok)
    for keep, first, last in ((0, 0, 0), (10, 6, 5), (10, -1, 0), (10, 0, -1)):
        with pytest.raises(SkvError):
            evict(c.ctx, c.rows, w, keep, first, last)
    for parts in (0, 9):
        with pytest.raises(ValueError):
            c.ctx.join([c.out] * parts, [c.lse] * parts, c.out, c.lse)
    assert c.ctx.get_device_error() == 0
    c.attend()
    c.check()


def test_a_set_error_word_leaves_nothing_kept():
    rows, w = _rows(1, 100), torch.rand((1, 100), device="cuda")
    with Context(Config(max_requests=1, num_layers=1, max_context=4, topk=1, hot_slots=1, max_batch=1)) as ctx:
        ids, one = torch.tensor([0], dtype=torch.int32, device="cuda"), torch.zeros((1, 1, 1), dtype=torch.int32, device="cuda")
        ctx.assemble(ids, one, one.clone(), one.clone(), one.clone())  # no such request
        kept, out, kw = evict(ctx, rows, w, 10)
        assert bool((kept == -1).all()) and bool((out == 7).all()) and bool((kw == 7).all())
        assert ctx.get_device_error() != 0
        check_evicted(rows, w, 10, 0, 0, evict(ctx, rows, w, 10))
