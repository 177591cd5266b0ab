"""Decode steps over a cache in 4 bits, as they are used: rows are packed and
published, each step selects its Top-k from the index keys, assembles the packed
rows, attends over them, and writes the next token back, against the definitions
(oracle/select.py, oracle/q4.py, oracle/attention.py); eagerly, as one captured
graph, and in two contexts side by side."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as g4
from oracle import attention as att
from oracle import q4
from oracle import select as sel

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import SKV_Q4_ROW_BYTES, Config, Context, Index

B, L, K, S, T0, STEPS, HEADS, DIM, BLOCK = 3, 2, 96, 160, 500, 4, 8, 64, 4
SCALE = 0.1


class Decode:
    """Buffers of a decode loop and one step of it."""

    def __init__(self, seed):
        rng = self.rng = np.random.default_rng(seed)
        T = T0 + STEPS + 2
        self.ctx = Context(Config(max_requests=B, num_layers=L, max_context=T, topk=K, hot_slots=S, max_batch=B,
                                  row_bytes=SKV_Q4_ROW_BYTES))
        # every row there will ever be, as bf16, and what the cache makes of it
        self.rows = g4._bf16((rng.standard_normal((B, L, T, 576)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16))
        flat = self.rows.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, 576)
        self.values = q4.values(q4.pack(g4._f64(flat))).reshape(B, L, T, 576)
        packed = torch.empty((L, T0, SKV_Q4_ROW_BYTES), dtype=torch.uint8, device="cuda")
        for b in range(B):
            self.ctx.pack_rows(self.rows[b, :, :T0].contiguous().view(-1, 576), packed)
            assert self.ctx.publish(T0, rows=packed) == b
            torch.cuda.synchronize()  # `packed` is used again
        n = -(-T // BLOCK)
        self.K = torch.from_numpy(sel.on_grid(rng, (B, L, n, DIM))).bfloat16().cuda()
        self.index = Index(self.K, block=BLOCK, first=1, last=2)
        self.req = torch.arange(B, dtype=torch.int32, device="cuda")
        self.qi = torch.empty((B, L, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        self.w = torch.empty((B, L, HEADS), device="cuda")
        self.q = torch.empty((B * L, 128, 576), dtype=torch.bfloat16, device="cuda")
        self.new = torch.empty((B, L, 576), dtype=torch.bfloat16, device="cuda")
        self.new_packed = torch.empty((B, L, SKV_Q4_ROW_BYTES), dtype=torch.uint8, device="cuda")
        self.topk = torch.empty((B, L, K), dtype=torch.int32, device="cuda")
        self.slots = torch.empty_like(self.topk)
        self.count = torch.empty((2, B, L), dtype=torch.int32, device="cuda")
        self.work = torch.empty(self.ctx.select_workspace(self.index, B), dtype=torch.uint8, device="cuda")
        self.out = torch.empty((B * L, 128, 512), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty((B * L, 128), device="cuda")
        self.len = T0

    def inputs(self):
        self.qi.copy_(torch.from_numpy(sel.on_grid(self.rng, (B, L, HEADS, DIM))))
        self.w.copy_(torch.from_numpy(self.rng.integers(-16, 65, (B, L, HEADS)) / 64))
        self.q.copy_(torch.from_numpy(self.rng.standard_normal((B * L, 128, 576))))
        self.new.copy_(self.rows[:, :, self.len])

    def step(self):
        c = self.ctx
        c.pack_rows(self.new.view(-1, 576), self.new_packed)
        c.write_back(self.req, self.new_packed)
        c.select(self.index, self.req, self.qi, self.w, self.topk, self.work)
        c.assemble(self.req, self.topk, self.slots, self.count[0], self.count[1])
        c.attend_q4(self.req, self.q, self.slots, self.out, self.lse, sm_scale=SCALE)

    def check(self):
        self.len += 1
        topk = self.topk.cpu().numpy()
        out = self.out.view(torch.int16).cpu().numpy().view(np.uint16)
        lse = self.lse.cpu().numpy()
        keys, qi, w, q = (t.double().cpu().numpy() for t in (self.K, self.qi, self.w, self.q))
        for b in range(B):
            for l in range(L):
                want = sel.select(keys[b, l], qi[b, l], w[b, l], self.len, K, BLOCK, 1, 2)
                assert np.array_equal(topk[b, l], want), (b, l)
                valid = want >= 0
                rows = np.zeros((K, 576))
                rows[valid] = self.values[b, l][want[valid]]
                o, s = att.attend(q[b * L + l], rows, valid, SCALE)
                lse_tol, atol, rtol = g4.ac.bounds(q[b * L + l], rows, valid, SCALE)
                got = g4._f64(out[b * L + l])
                assert np.all(np.abs(got - o) <= atol + (rtol + g4.ac.MISC) * np.abs(o)), (b, l)
                assert np.all(np.abs(lse[b * L + l] - s) <= lse_tol + g4.ac.MISC), (b, l)
        assert self.ctx.get_device_error() == 0


def test_decode_steps():
    d = Decode(1)
    for _ in range(STEPS):
        d.inputs()
        d.step()
        d.check()
    d.ctx.close()


def test_decode_steps_as_one_graph():
    d = Decode(2)
    d.inputs()
    d.step()
    d.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.step()
    for _ in range(STEPS - 1):
        d.inputs()
        g.replay()
        d.check()
    d.ctx.close()


def test_two_decodes_side_by_side():
    """Two contexts on two streams at the same time, one eager and one replayed."""
    a, b = Decode(3), Decode(4)
    b.inputs()
    b.step()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(STEPS - 1):
        a.inputs()
        b.inputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(sb):
            g.replay()
        with torch.cuda.stream(sa):
            a.step()
        torch.cuda.synchronize()
        a.check()
        b.check()
    a.ctx.close()
    b.ctx.close()


def test_layer_by_layer_on_another_stream():
    d = Decode(5)
    d.inputs()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    d.ctx.pack_rows(d.new.view(-1, 576), d.new_packed, stream=s)
    d.ctx.write_back(d.req, d.new_packed, stream=s)
    parts = []
    for l in range(L):
        topk = torch.empty((B, K), dtype=torch.int32, device="cuda")
        slots, n = torch.empty_like(topk), torch.empty((2, B), dtype=torch.int32, device="cuda")
        qi, w = d.qi[:, l].contiguous(), d.w[:, l].contiguous()
        q = d.q.view(B, L, 128, 576)[:, l].contiguous()
        out, lse = torch.empty((B, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 128), device="cuda")
        torch.cuda.synchronize()
        d.ctx.select(d.index, d.req, qi, w, topk, d.work, layer=l, stream=s)
        d.ctx.assemble_layer(l, d.req, topk, slots, n[0], n[1], stream=s)
        d.ctx.attend_q4(d.req, q, slots, out, lse, layer=l, sm_scale=SCALE, stream=s)
        s.synchronize()
        parts.append((topk, out, lse))
    d.topk.copy_(torch.stack([p[0] for p in parts], 1))
    d.out.copy_(torch.stack([p[1] for p in parts], 1).view_as(d.out))
    d.lse.copy_(torch.stack([p[2] for p in parts], 1).view_as(d.lse))
    d.check()
    d.ctx.close()
