"""Attention over a prefix where a cluster takes several items of the work, each call followed at once by kernels that
use the same shared memory."""
import pytest
import torch

from test_gpu_prefix import SCALE, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [4, 8, 0])
@pytest.mark.parametrize("B,L,n,heads", [(2, 1, 100, 128), (7, 3, 300, 128), (90, 2, 130, 128), (50, 3, 700, 40)])
def test_items_of_several_rounds_between_other_kernels(B, L, n, heads, sms):
    c = Case(B, L, n, heads, seed=n)
    c.ctx.set_attend_sms(sms)
    c.attend()
    c.check()
    lse, weights = c.lse[:-1].clone(), torch.empty((L, n), device="cuda")
    want = [c.out.clone(), c.lse.clone(), c.weigh(lse, None, out=weights).clone()]
    attend_work = torch.empty(c.ctx.attend_prefix_workspace(c.prefix, B, heads), dtype=torch.uint8, device="cuda")
    weigh_work = torch.empty(c.ctx.weigh_prefix_workspace(c.prefix, B, heads), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(20):
        c.out.fill_(7)
        c.lse.fill_(7)
        c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, attend_work, sm_scale=SCALE)
        c.ctx.weigh_prefix(c.prefix, c.q, lse, None, weights, weigh_work, sm_scale=SCALE)
        c.ctx.attend_prefix(c.prefix, c.q, c.out, c.lse, attend_work, sm_scale=SCALE)
        got.append([c.out.clone(), c.lse.clone(), weights.clone()])
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    assert c.ctx.get_device_error() == 0
