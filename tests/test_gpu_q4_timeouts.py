"""Waits of skv_attend_q4 and skv_select that run out, without harm to a GPU: the
loads are withheld, so nothing is in flight, and the kernels report SKV_DEVERR_TIMEOUT
and leave the context usable."""
import pytest
import torch

import test_gpu_q4 as g4
from test_gpu_select import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import skv


@pytest.mark.parametrize("B,L,k,sms", [(2, 2, 300, 2), (2, 2, 300, 0), (1, 1, 65, 0)])
def test_attention_whose_rows_never_come_reports_timeout(B, L, k, sms):
    """Several units a pair of SMs; units split over pairs (the joining kernel runs as well)."""
    c = g4.Cache(B, L, k + 50, k, seed=51, pad=3)
    out, lse = g4._outputs(B * L)
    c.ctx.set_attend_sms(sms)
    c.ctx.selftest_attend_timeout(c.req_dev, c.q_dev, c.slots, out)
    torch.cuda.synchronize()
    assert c.ctx.get_device_error() == skv.SKV_DEVERR_TIMEOUT
    assert c.ctx.get_device_error() == 0  # read and cleared
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, out, lse, sm_scale=0.1)
    c.check(out, lse, 0.1)
    assert c.ctx.get_device_error() == 0
    c.ctx.close()


@pytest.mark.parametrize("lens,T_max", [([900, 300, 64], None), ([40000, 20000], None), ([5, 9], 400000)])
def test_selection_whose_keys_never_come_reports_timeout(lens, T_max):
    """One CTA a unit; teams; rows that would need no scores."""
    c = Case(len(lens), 2, lens, 64, 8, 64, seed=52, T_max=T_max)
    out = torch.full((len(lens), 2, 64), -7, dtype=torch.int32, device="cuda")
    c.ctx.selftest_select_timeout(c.index, c.req_dev, c.q, c.w, out, c.work)
    torch.cuda.synchronize()
    assert bool((out == -1).all())
    assert bool((c.run() == -1).all())  # the word is sticky
    assert c.ctx.get_device_error() == skv.SKV_DEVERR_TIMEOUT
    c.check(c.run())
