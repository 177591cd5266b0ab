"""A prefix however its rows lie: token-major caches, layers padded by a part of a row, a single token, layers that share
memory.  What lies between the rows is NaN where nothing else needs it."""
import math

import pytest
import torch

from oracle import prefix as pre
from test_gpu_prefix import Case, _check_weights, check_evicted, evict

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Prefix, SkvError

# (layers, tokens, strides of a layer and of a row in values)
LAYOUTS = {
    "token-major": lambda L, n: (576, 576 * L),
    "token-major in wider rows": lambda L, n: (640, 640 * L + 24),
    "layers a part of a row apart": lambda L, n: (576 * n + 8, 576),
    "wider rows, layers on borders of 256 bytes": lambda L, n: ((640 * n + 72 + 127) // 128 * 128 + 128, 640 + 8),
    "layers a whole number of wide rows apart": lambda L, n: (584 * (n + 5), 584),
    "layers that share rows": lambda L, n: (600, 600),
    "layers that share parts of rows": lambda L, n: (584, 1160),
    "layers side by side in very wide rows": lambda L, n: (584, 2 ** 16 + 8),
}


def lay(c, layer, row):
    """The case's prefix at these strides."""
    L, n = c.L, c.n
    size = (L - 1) * layer + (n - 1) * row + 576
    g = torch.Generator(device="cuda").manual_seed(n)
    apart = layer >= (n - 1) * row + 576 or row >= (L - 1) * layer + 576
    flat = torch.full((size + 8,), math.nan, device="cuda", dtype=torch.bfloat16) if apart else \
        torch.randn(size + 8, generator=g, device="cuda").bfloat16()
    view = flat.as_strided((L, n, 576), (layer, row, 1))
    if apart:
        view.copy_(c.rows)
    c.rows, c.prefix = view, Prefix(view)
    return c


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("B,L,n,heads", [(2, 3, 1, 128), (3, 4, 2, 40), (5, 3, 130, 40), (2, 5, 1001, 128), (70, 2, 300, 128)])
def test_attention_weights_and_eviction_of_any_layout(name, B, L, n, heads):
    layer, row = LAYOUTS[name](L, n)
    c = lay(Case(B, L, n, heads, seed=n), layer, row)
    whole = c.attend()[0][:-1].clone()
    c.check()
    again = c.attend()[0][:-1]
    assert torch.equal(whole, again)
    lse, before = c.shares(), torch.rand((L, n), device="cuda")
    weights = c.weigh(lse, before)
    _check_weights(c, weights, lse, before)
    keep = max(1, n // 3)
    check_evicted(c.rows, weights, keep, 0, 1, evict(c.ctx, c.rows, weights, keep, 0, 1))
    q = c.q
    for l in range(L):  # a layer at a time
        c.q = q.view(B, L, heads, 576)[:, l].contiguous()
        out, got = c.attend(layer=l)
        want, want_lse, off, lse_off = pre.attend(c.q.flatten(0, 1), c.rows[l], 1.0 / 24.0)
        assert bool(((out[:B].flatten(0, 1).double() - want).abs() <= off).all())
        assert bool(((got[:B].flatten().double() - want_lse).abs() <= lse_off).all())
        one = torch.full_like(before, 9.0)
        c.weigh(lse.view(B, L, heads)[:, l].contiguous(), before, out=one, layer=l)
        want, off = pre.weigh(c.q.flatten(0, 1), c.rows[l], lse.view(B, L, heads)[:, l].flatten(), 1.0 / 24.0, before[l])
        assert bool(((one[l].double() - want).abs() <= off).all()) and bool((one[[x for x in range(L) if x != l]] == 9).all())
    assert c.ctx.get_device_error() == 0


def test_one_layer_in_wider_rows():
    c = Case(3, 1, 700, gap=72)
    c.attend()
    c.check()


def test_layouts_without_a_pause_and_in_a_graph():
    """Launches of several layers one after the other share the workspace."""
    c = lay(Case(3, 4, 2000, seed=1), 576 * 2000 + 8, 576)
    work = torch.empty(max(c.ctx.attend_prefix_workspace(c.prefix, 3), c.ctx.weigh_prefix_workspace(c.prefix, 3)), dtype=torch.uint8, device="cuda")
    weights = torch.zeros((4, 2000), device="cuda")

    def step():
        c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, work, sm_scale=1.0 / 24.0, B=3)
        c.ctx.weigh_prefix(c.prefix, c.q, c.lse[:-1], None, weights, work, sm_scale=1.0 / 24.0, B=3)

    step()
    torch.cuda.synchronize()
    c.check()
    want = [t.clone() for t in (c.out, c.lse, weights)]
    _check_weights(c, weights, c.lse[:-1], None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for t in (c.out, c.lse, weights):
        t.fill_(7)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.lse, weights)))
    assert c.ctx.get_device_error() == 0
    del graph


def test_an_empty_prefix_of_any_strides():
    c = Case(3, 2, 0)
    c.prefix = Prefix(torch.empty((4,), device="cuda", dtype=torch.bfloat16).as_strided((2, 0, 576), (8, 8, 1)))
    c.attend()
    c.check()


def test_a_workspace_of_another_layout_is_refused_where_it_is_too_small():
    c = Case(1, 8, 3000)
    planes = c.ctx.attend_prefix_workspace(c.prefix, 1)
    lay(c, 576 * 3000 + 8, 576)
    alone = c.ctx.attend_prefix_workspace(c.prefix, 1)
    assert planes != alone
    work = torch.full((alone + 64,), 99, device="cuda", dtype=torch.uint8)
    with pytest.raises(SkvError):
        c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, work[:alone - 16], sm_scale=1.0 / 24.0)
    c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, work[:alone], sm_scale=1.0 / 24.0)
    c.check()
    assert bool((work[alone:] == 99).all())
