"""Calls that follow one another on a stream without a pause, each reading what
the call before it wrote into buffers that are used again with other data.

pack, unpack, attend_q4 and select start while the kernel before them still runs,
and wait for it before they read.  Their inputs here come straight from such a
kernel; the results have to be those of the same calls with the device idle
between any two of them, bit for bit (the kernels always sum in the same order),
and for the rows those of the oracle."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as g4
from oracle import q4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import SKV_Q4_ROW_BYTES, Config, Context, Index

ROUNDS = 24


def _packed(n, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((n, 576)) * np.exp2(rng.uniform(-2, 2, 576))).astype(np.float32)
    return q4.pack(g4._f64((x.view(np.uint32) >> 16).astype(np.uint16)))


@pytest.mark.parametrize("n", [1, 40, 1536, 20000])
def test_pack_and_unpack_of_one_another(n):
    """rows -> packed -> values -> packed again, always in the same buffers."""
    src = [_packed(n, seed) for seed in range(4)]
    src_dev = [torch.from_numpy(p).cuda() for p in src]
    rows = torch.empty((n, 576), dtype=torch.bfloat16, device="cuda")
    packed = torch.empty((n, SKV_Q4_ROW_BYTES), dtype=torch.uint8, device="cuda")
    got = [torch.zeros_like(packed) for _ in range(ROUNDS)]
    back = [torch.zeros_like(rows) for _ in range(ROUNDS)]
    with g4._ctx() as ctx:
        torch.cuda.synchronize()
        for i in range(ROUNDS):
            ctx.unpack_rows(src_dev[i % 4], rows)
            ctx.pack_rows(rows, packed)           # reads what unpack has just written
            ctx.unpack_rows(packed, rows)         # overwrites what pack has just read
            ctx.pack_rows(rows, got[i], back[i])
        torch.cuda.synchronize()
        want = []
        for p in src:
            v = q4.values(q4.pack(q4.values(p)))
            want.append((q4.pack(v), q4.values(q4.pack(v))))
        for i in range(ROUNDS):
            w_packed, w_values = want[i % 4]
            assert np.array_equal(got[i].cpu().numpy(), w_packed), i
            g4._same_values(back[i].view(torch.int16).cpu().numpy().view(np.uint16), w_values)


@pytest.mark.parametrize("B,L,k", [(1, 1, 512), (6, 2, 200), (30, 4, 130)])
def test_attention_whose_queries_come_from_the_call_before(B, L, k):
    c = g4.Cache(B, L, k + 50, k, seed=3)
    units = B * L
    src = [torch.from_numpy(_packed(units * 128, 50 + i)).cuda() for i in range(3)]
    q = torch.empty((units * 128, 576), dtype=torch.bfloat16, device="cuda")

    def run(pause):
        outs = []
        for i in range(ROUNDS):
            outs.append(g4._outputs(units))
        torch.cuda.synchronize()
        for i in range(ROUNDS):
            c.ctx.unpack_rows(src[i % 3], q)
            pause()
            c.ctx.attend_q4(c.req_dev, q, c.slots, *outs[i], sm_scale=0.01)
            pause()
        torch.cuda.synchronize()
        return outs

    slow, fast = run(torch.cuda.synchronize), run(lambda: None)
    for i, (a, b) in enumerate(zip(slow, fast)):
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1]), i
    assert not torch.equal(slow[0][1], slow[1][1])
    c.ctx.close()


@pytest.mark.parametrize("T,k", [(300, 64), (5000, 256), (40000, 512)])
def test_selection_whose_queries_come_from_the_call_before(T, k):
    B, heads, dim = 2, 9, 64  # a row of 576 values is the query of nine heads
    rng = np.random.default_rng(T)
    keys = torch.from_numpy(rng.standard_normal((B, 1, T, dim))).to(torch.bfloat16).cuda()
    w = torch.from_numpy(rng.random((B, 1, heads))).float().cuda()
    src = [torch.from_numpy(_packed(B, 70 + i)).cuda() for i in range(3)]
    rows = torch.empty((B, 576), dtype=torch.bfloat16, device="cuda")
    with Context(Config(max_requests=B, num_layers=1, max_context=T, topk=k, hot_slots=k, max_batch=B, row_bytes=16)) as ctx:
        req = torch.tensor([ctx.publish(T) for _ in range(B)], dtype=torch.int32, device="cuda")
        ix = Index(keys)
        work = torch.empty(ctx.select_workspace(ix, B), dtype=torch.uint8, device="cuda")

        def run(pause):
            outs = [torch.full((B, 1, k), -7, dtype=torch.int32, device="cuda") for _ in range(ROUNDS)]
            torch.cuda.synchronize()
            for i in range(ROUNDS):
                ctx.unpack_rows(src[i % 3], rows)
                pause()
                ctx.select(ix, req, rows.view(B, 1, heads, dim), w, outs[i], work)
                pause()
            torch.cuda.synchronize()
            return outs

        slow, fast = run(torch.cuda.synchronize), run(lambda: None)
        for i, (a, b) in enumerate(zip(slow, fast)):
            assert torch.equal(a, b), i
        assert not torch.equal(slow[0], slow[1]) and ctx.get_device_error() == 0
