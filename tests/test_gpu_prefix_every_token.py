"""Attention over long prefixes and the weights of their tokens, token by token: every marked token has a value dim and a
head's class of its own, so one that is dropped, read twice or taken from another place shows.  And the eviction of long
rows in a graph.

A token of class c holds 8 in rope dim 512 + c, and so does every query of that class in its own; all scores are 64 or 0,
and what is not marked has e^-64 of a marked token's share.  P of a marked token is 1 but for 2^-17 or so (the
score's log2, 92.3, is rounded to 2^-18), which bf16 rounds to 1, so with m tokens in a class
    out = 1 / m in each token's dim:  off by the output's rounding to bf16 (2^-8) and by 2^-12 for the joining of splits;
    lse = 64 + log m:  four roundings to 2^-18 of numbers up to 101 in log2, two that the joining adds, and log2 e and
          ln 2 in fp32 (101 * 2^-24 each): under 4e-5, where a token of a class of 512 is 2e-3;
    a weight = (heads of the class) / m:  off by 1e-4 of itself, twice the lse's bound and the exponent's own rounding."""
import math

import pytest
import torch

from test_gpu_prefix import _rows, context, evict

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Prefix

CLASSES, DIMS = 64, 512


def check_tokens(B, L, n, heads, marked, sms=0):
    """marked: tokens, ascending, at most CLASSES * DIMS of them."""
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = torch.randn((L, n, 576), generator=g, device="cuda", dtype=torch.bfloat16)
    rows[..., 512:] = 0
    k = torch.arange(len(marked), device="cuda")
    order = torch.stack([torch.randperm(len(marked), generator=g, device="cuda") for _ in range(L)])  # of marked, a layer
    for l in range(L):
        at = marked[order[l]]
        rows[l, at] = 0
        rows[l, at, 512 + k % CLASSES] = 8
        rows[l, at, k // CLASSES] = 1
    cls = torch.randint(CLASSES, (B * L, heads), generator=g, device="cuda")
    q = torch.zeros((B * L, heads, 576), device="cuda", dtype=torch.bfloat16)
    q.scatter_(2, 512 + cls[..., None], 8.0)
    count = torch.bincount(k % CLASSES, minlength=CLASSES)
    assert int(count.min()) > 0
    out, lse = torch.empty((B * L, heads, 512), device="cuda", dtype=torch.bfloat16), torch.empty((B * L, heads), device="cuda")
    weights, prefix = torch.empty((L, n), device="cuda"), Prefix(rows)
    with context(B, L) as ctx:
        ctx.set_attend_sms(sms)
        work = torch.empty(max(ctx.attend_prefix_workspace(prefix, B, heads), ctx.weigh_prefix_workspace(prefix, B, heads)),
                           dtype=torch.uint8, device="cuda")
        ctx.attend_prefix(prefix, q, out, lse, work, sm_scale=1.0)
        ctx.weigh_prefix(prefix, q, lse, None, weights, work, sm_scale=1.0)
        assert ctx.get_device_error() == 0
    m = count[cls].double()
    assert bool(((lse.double() - 64 - m.log()).abs() <= 4e-5).all()), float((lse.double() - 64 - m.log()).abs().max())
    want = (torch.arange(DIMS, device="cuda") < m[..., None]).double() / m[..., None]
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -12) * want + 1e-20).all())
    for l in range(L):
        taken = torch.bincount(cls.view(B, L, heads)[:, l].flatten(), minlength=CLASSES)
        full = torch.zeros(n, dtype=torch.float64, device="cuda")
        full[marked[order[l]]] = (taken / count)[k % CLASSES].double()
        assert bool(((weights[l].double() - full).abs() <= 1e-4 * full + 1e-20).all())


@pytest.mark.parametrize("B,L,n,heads,sms", [
    (1, 1, 32768, 64, 0), (1, 1, 32767, 128, 0), (1, 2, 20001, 16, 0), (3, 1, 5003, 128, 4), (3, 3, 5003, 40, 0), (80, 1, 4097, 128, 0),
    (37, 2, 1500, 128, 0), (5, 1, 30001, 128, 20)])
def test_every_token_counts_once(B, L, n, heads, sms):
    check_tokens(B, L, n, heads, torch.arange(n, device="cuda"), sms)


@pytest.mark.parametrize("B,heads", [(1, 8), (2, 128)])
def test_tokens_all_over_a_prefix_beyond_four_gigabytes(B, heads):
    """32768 of 3.9 million: evenly spread, in the first and the last block, and in a run across 4 GB."""
    n, across = 3_900_001, 2 ** 32 // 1152
    spread = torch.arange(30000, device="cuda") * n // 30000
    runs = [torch.arange(a, b, device="cuda") for a, b in ((0, 130), (n - 130, n), (across - 500, across + 500), (2 ** 31 // 1152 - 300, 2 ** 31 // 1152 + 300))]
    check_tokens(B, 1, n, heads, torch.cat((spread, *runs)).unique()[:CLASSES * DIMS])


def test_eviction_of_long_rows_in_graphs():
    """Two graphs with a workspace each, replayed on two streams with weights that change."""
    n, keep = 70001, 20000
    rows = _rows(2, n, 0)
    with context(L=2) as ctx:
        prefix, graphs = Prefix(rows), []
        for _ in range(2):
            w, kept = torch.rand((2, n), device="cuda"), torch.empty((2, keep), dtype=torch.int32, device="cuda")
            out, kw = torch.empty((2, keep, 576), device="cuda", dtype=torch.bfloat16), torch.empty((2, keep), device="cuda")
            work = torch.full((ctx.evict_prefix_workspace(prefix),), 0xA5, dtype=torch.uint8, device="cuda")
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ctx.evict_prefix(prefix, w, kept, out, kw, work, first=3, last=5)
            graphs.append((graph, torch.cuda.Stream(), w, kept, out, kw))
        for i in range(4):
            for j, (_, _, w, *_) in enumerate(graphs):
                w.copy_(torch.exp(3 * torch.randn((2, n), device="cuda")) if i % 2 else (torch.rand((2, n), device="cuda") > 0.8 - 0.1 * j).float())
            torch.cuda.synchronize()
            for graph, stream, *_ in graphs:
                with torch.cuda.stream(stream):
                    graph.replay()
                    graph.replay()
            torch.cuda.synchronize()
            for _, _, w, kept, out, kw in graphs:
                want = evict(ctx, rows, w, keep, 3, 5)
                best = w.clone()
                best[:, :3] = best[:, n - 5:] = math.inf
                at = torch.sort(best, descending=True, stable=True)[1][:, :keep].sort()[0]
                assert torch.equal(kept.long(), at) and torch.equal(kept, want[0])
                assert torch.equal(out.view(torch.int16), want[1].view(torch.int16)) and torch.equal(kw, want[2])
        assert ctx.get_device_error() == 0
        del graphs
