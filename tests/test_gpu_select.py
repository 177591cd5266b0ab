"""skv_select against its definition.

On values of a coarse grid every product and sum is exact in fp32 whatever
the order, so the selection has to equal the float64 one entry for entry,
ties included (there are many).  On arbitrary values two scores that differ
by less than their rounding may come in either order: each product is exact in
fp32, the sums have dim + heads terms, each rounding is at most 2^-22 of the
magnitudes summed (as in tests/test_gpu_attention.py), so no taken block may score
lower than one left out by more than
    2 * (dim / 16 + heads + 4) * 2^-22 * sum_h |w_h| sum_d |q_hd k_jd|.
"""
import numpy as np
import pytest
import torch

import oracle as orc
from oracle import select as sel

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Config, Context, Index, SkvError, skv


class Case:
    def __init__(self, B, L, lens, k, heads, dim, block=1, first=0, last=0, relu=True, T_max=None, R=None, seed=1,
                 grid=True, layout="rlnd"):
        rng = np.random.default_rng(seed)
        self.__dict__.update(B=B, L=L, k=k, heads=heads, dim=dim, block=block, first=first, last=last, relu=relu)
        R = R or B
        T_max = T_max or max(max(lens), 1)
        n = -(-T_max // block)
        self.ctx = Context(Config(max_requests=R, num_layers=L, max_context=T_max, topk=k, hot_slots=k, max_batch=B,
                                  row_bytes=16))
        self.req = [int(r) for r in rng.permutation(R)[:B]]
        self.lens = [0] * R
        for b, r in enumerate(self.req):
            self.lens[r] = lens[b]
        for r in range(R):
            assert self.ctx.publish(self.lens[r]) == r
        draw = sel.on_grid if grid else (lambda g, s: g.standard_normal(s))
        self.K = torch.from_numpy(draw(rng, (R, L, n, dim))).bfloat16().cuda()
        self.q = torch.from_numpy(draw(rng, (B, L, heads, dim))).bfloat16().cuda()
        self.w = torch.from_numpy(rng.integers(-16, 65, (B, L, heads)) / 64).float().cuda()
        order = ["rlnd".index(a) for a in layout[:3]]
        self.Kd = self.K.permute(*order, 3).contiguous().permute(*[order.index(i) for i in range(3)], 3)
        assert torch.equal(self.Kd, self.K)
        self.req_dev = torch.tensor(self.req, dtype=torch.int32, device="cuda")
        self.index = Index(self.Kd, block=block, first=first, last=last, relu=relu)
        self.work = torch.full((self.ctx.select_workspace(self.index, B),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, layer=-1):
        q, w = (self.q, self.w) if layer < 0 else (self.q[:, layer].contiguous(), self.w[:, layer].contiguous())
        out = torch.full((self.B, self.L, self.k) if layer < 0 else (self.B, self.k), -7, dtype=torch.int32, device="cuda")
        self.ctx.select(self.index, self.req_dev, q, w, out, self.work, layer=layer)
        return out

    def want(self, b, l):
        r = self.req[b]
        K, q, w = (t.double().cpu().numpy() for t in (self.K[r, l], self.q[b, l], self.w[b, l]))
        return sel.select(K, q, w, self.lens[r], self.k, self.block, self.first, self.last, self.relu)

    def check(self, out, layer=-1):
        out = out.cpu().numpy()
        for b in range(self.B):
            for l in range(self.L) if layer < 0 else [layer]:
                got = out[b, l] if layer < 0 else out[b]
                assert np.array_equal(got, self.want(b, l)), (b, l)
        assert self.ctx.get_device_error() == 0
        self.ctx.close()


@pytest.mark.parametrize("heads,dim,relu", [(1, 64, True), (1, 128, False), (7, 64, False), (16, 128, True), (17, 64, True),
                                            (32, 128, True), (37, 128, False), (48, 64, True), (64, 128, True), (64, 64, False)])
def test_heads_and_dims(heads, dim, relu):
    c = Case(3, 2, [1000, 333, 700], 64, heads, dim, relu=relu, seed=heads)
    c.check(c.run())


@pytest.mark.parametrize("lens", [[1], [2], [63], [64], [65], [127], [128], [129], [255], [257], [2047], [2048], [4097],
                                  [0, 1, 64, 65, 0], [0], [5000, 3, 0, 129, 64]])
def test_lengths(lens):
    """Lengths around k, around a tile of 128 keys, and of zero."""
    c = Case(len(lens), 2, lens, 64, 8, 64, seed=len(lens) + lens[0], T_max=max(lens) + 3, R=len(lens) + 1)
    c.check(c.run())


@pytest.mark.parametrize("block,k,first,last", [(1, 1, 0, 0), (1, 300, 5, 7), (1, 8, 4, 4), (2, 64, 0, 0), (16, 64, 1, 1), (16, 64, 0, 4),
                                                (64, 64, 0, 1), (64, 256, 2, 0), (100, 300, 0, 0), (128, 128, 0, 0)])
def test_blocks_and_forced_ends(block, k, first, last):
    c = Case(4, 2, [3001, 1, 640, 101], k, 16, 64, block=block, first=first, last=last, relu=False, seed=block)
    c.check(c.run())


@pytest.mark.parametrize("layout", ["rlnd", "rnld", "lrnd", "nrld", "lnrd"])
def test_index_layouts(layout):
    c = Case(3, 3, [300, 200, 129], 32, 8, 128, layout=layout, seed=3, R=4)
    c.check(c.run())


@pytest.mark.parametrize("B,L,ctx,k", [(1, 1, 20000, 2048), (2, 2, 70000, 512), (1, 1, 300000, 2048), (1, 1, 24576, 100),
                                       (1, 1, 24577, 100), (160, 1, 3000, 256), (40, 4, 1500, 64)])
def test_long_contexts_and_many_units(B, L, ctx, k):
    """Teams of 1 to 8 CTAs, scores kept in shared memory and not."""
    c = Case(B, L, [ctx - 7 * b for b in range(B)], k, 4, 64, seed=ctx)
    c.check(c.run())


def test_one_layer():
    c = Case(5, 3, [900, 1, 130, 70, 500], 64, 12, 64, seed=4)
    c.check(c.run(layer=2), layer=2)


def test_equal_scores_go_to_the_lower_index():
    c = Case(2, 1, [5000, 40000], 777, 4, 64, seed=5)
    c.K.zero_()
    c.K[:, :, 1000:1100] = 1.0  # one hundred better than the rest, all alike
    c.Kd.copy_(c.K)
    c.q.fill_(1.0)
    c.w.fill_(1.0)
    out = c.run().cpu().numpy()
    want = np.r_[0:677, 1000:1100]
    assert np.array_equal(out[0, 0], want) and np.array_equal(out[1, 0], want)
    c.check(c.run())


@pytest.mark.parametrize("relu", [True, False])
def test_infinities_nans_and_what_lies_behind_the_length(relu):
    c = Case(2, 1, [700, 900], 64, 4, 64, relu=relu, seed=6, T_max=1000)
    for r, t in zip(c.req, (700, 900)):
        c.K[r, 0, t:] = float("nan")   # behind the request's last key
        c.K[r, 0, 10] = float("nan")
        c.K[r, 0, 11, 5] = float("inf")
        c.K[r, 0, 12, 5] = float("-inf")
        c.K[r, 0, 13] = 3e38
    c.q[:, :, :, 5] = 1.0
    c.q[:, :, 2, 7:] = 0.0
    c.w.abs_().add_(1 / 64)
    c.Kd.copy_(c.K)
    out = c.run().cpu().numpy()
    for b, (r, T) in enumerate(zip(c.req, (700, 900))):
        got = set(out[b, 0])
        # the float64 scores, with what overflows 32 bits as infinities
        s = sel.scores(*(t.double().cpu().numpy() for t in (c.K[r, 0], c.q[b, 0], c.w[b, 0])), relu)
        plain = np.ones(1000, bool)
        plain[10:14] = False
        assert 11 in got and (relu or 10 not in got) and max(got) < T
        others = np.array([j for j in range(T) if plain[j]])
        left = 64 - len(got & {10, 11, 12, 13})
        best = set(others[np.lexsort((others, -s[others]))][:left])
        assert got - {10, 11, 12, 13} == best
    assert c.ctx.get_device_error() == 0
    c.ctx.close()


@pytest.mark.parametrize("seed", range(3))
def test_arbitrary_values_within_rounding(seed):
    c = Case(4, 2, [3000, 2500, 640, 2999], 300, 64, 128, grid=False, seed=seed)
    out = c.run().cpu().numpy()
    for b, r in enumerate(c.req):
        for l in range(2):
            K, q, w = (t.double().cpu().numpy()[:c.lens[r]] for t in (c.K[r, l], c.q[b, l], c.w[b, l]))
            s = sel.scores(K, q, w, True)
            err = 2 * (128 / 16 + 64 + 4) * 2.0 ** -22 * (np.abs(w) @ (np.abs(q) @ np.abs(K).T)).max()
            got = out[b, l]
            assert np.all(np.diff(got) > 0) and got[0] >= 0 and got[-1] < c.lens[r]
            left = np.setdiff1d(np.arange(c.lens[r]), got)
            assert s[got].min() >= s[left].max() - err
    c.ctx.close()


def test_same_bits_again_in_a_graph_and_after_the_lengths_grew():
    c = Case(3, 2, [500, 64, 200], 64, 8, 64, T_max=600, seed=8)
    first = c.run()
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.ctx.select(c.index, c.req_dev, c.q, c.w, out, c.work)
    g.replay()
    assert torch.equal(out, first)
    rows = torch.zeros((2, 37, 16), dtype=torch.uint8, device="cuda")
    for r in c.req:  # the captured call reads the lengths when it runs
        c.ctx.extend(r, rows, 37)
        c.lens[r] += 37
    g.replay()
    c.check(out)


def test_two_graphs_with_a_workspace_each_side_by_side():
    a = Case(2, 1, [4000, 3000], 64, 8, 64, seed=9)
    b = Case(2, 1, [2000, 3500], 64, 8, 64, seed=10)
    outs = [torch.empty((2, 1, 64), dtype=torch.int32, device="cuda") for _ in range(2)]
    graphs = []
    for c, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.ctx.select(c.index, c.req_dev, c.q, c.w, o, c.work)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_the_same_request_twice():
    c = Case(2, 1, [800, 900], 64, 8, 64, seed=11)
    c.req = [c.req[0], c.req[0]]
    c.req_dev = torch.tensor(c.req, dtype=torch.int32, device="cuda")
    c.check(c.run())


def test_bad_requests_fill_the_call_with_minus_one():
    c = Case(3, 2, [800, 900, 100], 64, 8, 64, seed=12, R=4)
    other = next(r for r in range(4) if r not in c.req)
    c.ctx.release(other)
    good = c.req_dev
    for ids in ([c.req[0], -1, c.req[2]], [c.req[0], 4, c.req[2]], [other, c.req[1], c.req[2]]):
        c.req_dev = torch.tensor(ids, dtype=torch.int32, device="cuda")
        assert bool((c.run() == -1).all())
        c.req_dev = good
        assert bool((c.run() == -1).all())  # the error word is sticky
        assert c.ctx.get_device_error() == orc.E_BAD_REQUEST
    c.check(c.run())


def test_refuses_bad_arguments():
    c = Case(2, 2, [300, 200], 64, 8, 64, block=2, seed=13)
    out = torch.full((2, 2, 64), -7, dtype=torch.int32, device="cuda")
    bad = skv.SKV_ERR_INVALID_ARG
    base = dict(keys=c.Kd.data_ptr(), request_stride=2 * c.Kd.stride(0), layer_stride=2 * c.Kd.stride(1),
                key_stride=2 * c.Kd.stride(2), heads=8, dim=64, block=2, first=1, last=1, relu=1)
    args = [c.req_dev.data_ptr(), 2, -1, c.q.data_ptr(), c.w.data_ptr(), out.data_ptr(), c.work.data_ptr(), c.work.numel(), 0]

    def call(ix=None, **at):
        a = list(args)
        for i, v in at.items():
            a[int(i[1:])] = v
        return skv.skv_select(c.ctx.h, skv.ctypes.byref(skv.skv_index(**dict(base, **(ix or {})))), *a)

    for ix in (dict(keys=0), dict(keys=base["keys"] + 2), dict(heads=0), dict(heads=65), dict(dim=96), dict(dim=0), dict(block=0),
               dict(block=3), dict(block=128), dict(first=-1), dict(last=-1), dict(first=20, last=13), dict(key_stride=126),
               dict(key_stride=112), dict(key_stride=0), dict(key_stride=136), dict(layer_stride=0), dict(layer_stride=-128),
               dict(request_stride=8), dict(request_stride=1 << 40), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert call(ix) == bad, ix
    for at in (dict(_0=0), dict(_1=-1), dict(_1=3), dict(_2=-2), dict(_2=2), dict(_3=0), dict(_3=args[3] + 8), dict(_4=0), dict(_5=0),
               dict(_6=0), dict(_6=args[6] + 4), dict(_7=args[7] - 1), dict(_7=-1)):
        assert call(**at) == bad, at
    assert skv.skv_select(None, None, *args) == bad and skv.skv_select(c.ctx.h, None, *args) == bad
    assert call(_1=0, _0=0) == skv.SKV_OK
    n = skv.ctypes.c_int64(-5)
    assert skv.skv_select_workspace(c.ctx.h, None, 2, -1, skv.ctypes.byref(n)) == bad
    assert skv.skv_select_workspace(c.ctx.h, c.index.c(), 3, -1, skv.ctypes.byref(n)) == bad and n.value == -5
    with pytest.raises(ValueError):
        c.ctx.select(Index(c.Kd[:1], block=2), c.req_dev, c.q, c.w, out, c.work)  # fewer requests than the context
    with pytest.raises(ValueError):
        c.ctx.select(c.index, c.req_dev, c.q[..., :32], c.w, out, c.work)
    with pytest.raises(ValueError):
        c.ctx.select(c.index, c.req_dev, c.q, c.w[:1], out, c.work)
    with pytest.raises(ValueError):
        Index(c.Kd[0])
    with pytest.raises(SkvError):
        c.ctx.select(c.index, c.req_dev, c.q, c.w, out, c.work[:-16])
    torch.cuda.synchronize()
    assert bool((out == -7).all())
    c.ctx.close()
