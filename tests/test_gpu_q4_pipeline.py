"""A decode step layer by layer over a cache in 4 bits, with each layer's attention on
a stream of its own beside the next layer's selection and assembly: the same bits as
the layers one after the other."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as g4
from oracle import q4
from oracle import select as sel

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import SKV_Q4_ROW_BYTES, Config, Context, Index


class Layers:
    def __init__(self, B, L, T, k, S, sms):
        rng = np.random.default_rng(B * L)
        self.B, self.L = B, L
        self.ctx = Context(Config(max_requests=B, num_layers=L, max_context=T, topk=k, hot_slots=S, max_batch=B,
                                  row_bytes=SKV_Q4_ROW_BYTES))
        rows = q4.pack(rng.standard_normal((T, 576)))
        for b in range(B):  # each request and layer holds the rows in an order of its own
            self.ctx.publish(T, rows=np.stack([rows[rng.permutation(T)] for _ in range(L)]))
        self.index = Index(torch.from_numpy(sel.on_grid(rng, (B, L, T, 64))).bfloat16().cuda())
        self.req = torch.arange(B, dtype=torch.int32, device="cuda")
        self.work = torch.empty(self.ctx.select_workspace(self.index, B, layer=0), dtype=torch.uint8, device="cuda")
        self.ctx.set_attend_sms(sms)
        self.qi = torch.from_numpy(sel.on_grid(rng, (L, B, 8, 64))).bfloat16().cuda()
        self.w = torch.rand((L, B, 8), device="cuda")
        self.q = torch.randn((L, B, 128, 576), device="cuda").bfloat16()
        self.k = k

    def buffers(self):
        B, L, k = self.B, self.L, self.k
        return [(torch.empty((B, k), dtype=torch.int32, device="cuda"), torch.empty((B, k), dtype=torch.int32, device="cuda"),
                 torch.empty((2, B), dtype=torch.int32, device="cuda"), *g4._outputs(B)) for _ in range(L)]

    def step(self, bufs, first, second, qi):
        """Selection and assembly on `first`, attention on `second`."""
        for l, (topk, slots, n, out, lse) in enumerate(bufs):
            self.ctx.select(self.index, self.req, qi[l], self.w[l], topk, self.work, layer=l, stream=first)
            self.ctx.assemble_layer(l, self.req, topk, slots, n[0], n[1], stream=first)
            second.wait_stream(first)
            self.ctx.attend_q4(self.req, self.q[l], slots, out, lse, layer=l, sm_scale=0.1, stream=second)
        first.wait_stream(second)


@pytest.mark.parametrize("B,L,T,k,S,sms", [(3, 4, 900, 200, 300, 0), (3, 4, 900, 200, 300, 72), (96, 3, 1500, 512, 700, 72)])
def test_attention_beside_the_next_layers_selection_and_assembly(B, L, T, k, S, sms):
    d = Layers(B, L, T, k, S, sms)
    queries = [d.qi, -d.qi, d.qi.flip(0), d.qi.flip(1)]
    results = []
    for pipelined in (False, True):
        steps = [d.buffers() for _ in queries]
        torch.cuda.synchronize()
        one, two = torch.cuda.Stream(), torch.cuda.Stream()
        for bufs, qi in zip(steps, queries):
            d.step(bufs, one, two if pipelined else one, qi)
        torch.cuda.synchronize()
        assert d.ctx.get_device_error() == 0
        results.append(steps)
    for a, b in zip(*results):
        for l in range(L):
            assert torch.equal(a[l][0], b[l][0])  # the selection (its rows may lie in other slots the second time)
            assert torch.equal(a[l][3].view(torch.int16), b[l][3].view(torch.int16)) and torch.equal(a[l][4], b[l][4]), l
            assert not torch.isnan(a[l][4]).any()
    d.ctx.close()
