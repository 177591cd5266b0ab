"""Rows in 4 bits on the GPU: skv_pack_rows / skv_unpack_rows bit for bit
against the oracle, and skv_attend_q4 against the float64 attention over the
values its packed hot rows stand for.

The attention's tolerances are those of tests/attention_check.py: packed rows
become bf16 exactly, so the products, their accumulation and the exchange
between the two CTAs are skv_attend's.  A unit whose keys are split adds, per
split and for the join, one more ex2 / log2f / division of the kind that MISC
covers (relative errors of 2^-22 each) and fp32 sums over at most 64 splits:
one more MISC, on lse and on out.
"""
import numpy as np
import pytest
import torch

import attention_check as ac
from oracle import attention as att
from oracle import q4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import SKV_Q4_ROW_BYTES, Config, Context, SkvError, skv

ROW = 336


def _ctx(R=1, L=1, T=1, k=1, S=1, B=1, row_bytes=ROW):
    return Context(Config(max_requests=R, num_layers=L, max_context=T, topk=k, hot_slots=S, max_batch=B,
                          row_bytes=row_bytes))


def _bits(n, seed=1):
    return q4.test_rows(n, seed)


def _f64(bits):
    return att.bf16_rows_to_f64(bits.view(np.uint8))


def _bf16(bits):
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def _same_values(got_bits, want):
    """bf16 bits equal the float64 values (any NaN for a NaN)."""
    f = _f64(got_bits)
    assert np.array_equal(np.isnan(f), np.isnan(want))
    keep = ~np.isnan(want)
    assert np.array_equal(f[keep], want[keep])


@pytest.mark.parametrize("n", [1, 2, 7, 31, 32, 33, 64, 1000])
@pytest.mark.parametrize("stride", [576, 584, 640])
def test_pack_is_the_oracle_bit_for_bit(n, stride):
    bits = _bits(n, seed=n)
    want = q4.pack(_f64(bits))
    wide = torch.full((n, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :576] = _bf16(bits)
    packed = torch.full((n + 1, ROW), 0xA5, dtype=torch.uint8, device="cuda")
    values = torch.full((n + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    with _ctx() as ctx:
        ctx.pack_rows(wide[:, :576], packed, values)
        assert np.array_equal(packed[:n].cpu().numpy(), want)
        _same_values(values[:n].view(torch.int16).cpu().numpy().view(np.uint16), q4.values(want))
        # rows behind the last one are left as they were
        assert bool((packed[n] == 0xA5).all()) and bool((values[n] == 7.0).all())
        packed.fill_(0x5A)
        ctx.pack_rows(wide[:, :576], packed)  # without values
        assert np.array_equal(packed[:n].cpu().numpy(), want) and bool((packed[n] == 0x5A).all())


@pytest.mark.parametrize("n", [1, 3, 14, 15, 100, 1000])
def test_unpack_reads_what_a_packed_row_stands_for(n):
    want = q4.pack(_f64(_bits(n, seed=100 + n)))
    packed = torch.from_numpy(want).cuda()
    values = torch.full((n + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    with _ctx() as ctx:
        ctx.unpack_rows(packed, values)
        _same_values(values[:n].view(torch.int16).cpu().numpy().view(np.uint16), q4.values(want))
        assert bool((values[n] == 7.0).all())


@pytest.mark.parametrize("rows_at,values_at,stride", [(0, 0, 576), (8, 0, 576), (0, 8, 576), (8, 8, 584), (0, 0, 584), (0, 0, 592)])
def test_pack_and_unpack_at_16_and_32_byte_alignment(rows_at, values_at, stride):
    n = 77
    bits = _bits(n, seed=7)
    want = q4.pack(_f64(bits))
    buf = torch.zeros(n * stride + 64, dtype=torch.bfloat16, device="cuda")
    rows = buf[rows_at:rows_at + n * stride].view(n, stride)[:, :576]
    rows.copy_(_bf16(bits))
    packed = torch.zeros(n * ROW + 64, dtype=torch.uint8, device="cuda")[16:16 + n * ROW].view(n, ROW)
    out = torch.zeros(n * 576 + 64, dtype=torch.bfloat16, device="cuda")
    values = out[values_at:values_at + n * 576].view(n, 576)
    with _ctx() as ctx:
        ctx.pack_rows(rows, packed, values)
        assert np.array_equal(packed.cpu().numpy(), want)
        _same_values(values.view(torch.int16).cpu().numpy().view(np.uint16), q4.values(want))
        assert not out[:values_at].any() and not out[values_at + n * 576:].any()
        out.zero_()
        ctx.unpack_rows(packed, values)
        _same_values(values.view(torch.int16).cpu().numpy().view(np.uint16), q4.values(want))
        assert not out[:values_at].any() and not out[values_at + n * 576:].any()


def test_every_code_and_scale_unpacks_exactly():
    """All 16 codes under all e4m3 scales, at the ends of the exponent's range."""
    for e in (27, 127, 243):
        p = np.zeros((8, ROW), np.uint8)
        p[:, :288] = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], np.uint8), 36)
        p[:, 288:324] = (np.arange(8 * 36).reshape(8, 36) % 256).astype(np.uint8)
        p[:, 324] = e
        want = q4.values(p)
        values = torch.empty((8, 576), dtype=torch.bfloat16, device="cuda")
        with _ctx() as ctx:
            ctx.unpack_rows(torch.from_numpy(p).cuda(), values)
        _same_values(values.view(torch.int16).cpu().numpy().view(np.uint16), want)


def test_pack_to_pinned_memory_on_another_stream_and_in_a_graph():
    bits = _bits(50, seed=5)
    want = q4.pack(_f64(bits))
    rows = _bf16(bits)
    pinned = torch.zeros((50, ROW), dtype=torch.uint8).pin_memory()
    packed = torch.zeros((50, ROW), dtype=torch.uint8, device="cuda")
    back = torch.zeros((50, 576), dtype=torch.bfloat16, device="cuda")
    with _ctx() as ctx:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ctx.pack_rows(rows, pinned, stream=s)
        s.synchronize()
        assert np.array_equal(pinned.numpy(), want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.pack_rows(rows, packed)
            ctx.unpack_rows(packed, back)
        packed.zero_()
        rows.copy_(_bf16(_bits(50, seed=6)))
        g.replay()
        torch.cuda.synchronize()
        want = q4.pack(_f64(_bits(50, seed=6)))
        assert np.array_equal(packed.cpu().numpy(), want)
        _same_values(back.view(torch.int16).cpu().numpy().view(np.uint16), q4.values(want))


def test_pack_and_unpack_refuse_bad_arguments():
    rows = torch.zeros((4, 640), dtype=torch.bfloat16, device="cuda")
    packed = torch.zeros((5, ROW), dtype=torch.uint8, device="cuda")
    values = torch.zeros((5, 576), dtype=torch.bfloat16, device="cuda")
    r, p, v = rows.data_ptr(), packed.data_ptr(), values.data_ptr()
    with _ctx() as ctx:
        bad = skv.SKV_ERR_INVALID_ARG
        for args in ((r + 2, 1280, 4, p, v), (r, 1280, 4, p + 8, v), (r, 1280, 4, p, v + 2), (r, 1144, 4, p, v),
                     (r, 1160, 4, p, v), (r, 0, 4, p, v), (r, (1 << 24) + 16, 4, p, v), (r, 1280, -1, p, v),
                     (r, 1280, (1 << 32) + 1, p, v), (0, 1280, 4, p, v), (r, 1280, 4, 0, v)):
            assert skv.skv_pack_rows(ctx.h, *args, 0) == bad, args
        for args in ((p + 4, 4, v), (p, 4, v + 4), (0, 4, v), (p, 4, 0), (p, -1, v), (p, (1 << 32) + 1, v)):
            assert skv.skv_unpack_rows(ctx.h, *args, 0) == bad, args
        assert skv.skv_pack_rows(ctx.h, 0, 0, 0, 0, 0, 0) == skv.SKV_OK  # nothing to do
        assert skv.skv_unpack_rows(ctx.h, 0, 0, 0, 0) == skv.SKV_OK
        with pytest.raises(ValueError):
            ctx.pack_rows(rows, packed)  # 640 wide
        with pytest.raises(ValueError):
            ctx.pack_rows(rows[:, :576], packed[:3])
        with pytest.raises(ValueError):
            ctx.pack_rows(rows[:, :576].float(), packed)
        with pytest.raises(ValueError):
            ctx.unpack_rows(packed, values[:4])
        with pytest.raises(SkvError):
            ctx.pack_rows(rows[:1, :576].expand(4, 576), packed)  # rows on top of one another
        torch.cuda.synchronize()
        assert not packed.any()


# ------------------------------------------------------------------ attention
class Cache:
    """A context of packed rows with its requests published and one step assembled."""

    def __init__(self, B, L, T, k, seed, pad=0, S=None, R=None):
        self.B, self.L, self.k = B, L, k
        R = R or B
        rng = np.random.default_rng(seed)
        self.ctx = _ctx(R, L, T, k, S or max(k, 1), B)
        bits = np.stack([q4.test_rows(1, seed + 7 * r)[0] for r in range(R * L * 2)])
        x = rng.standard_normal((R, L, T, 576)) * np.exp2(rng.uniform(-1, 1, 576))
        x[0, 0, :1] = _f64(bits[:1])
        self.packed = q4.pack(x.reshape(-1, 576).astype(np.float32)).reshape(R, L, T, ROW)
        order = rng.permutation(R)[:B]
        ids = [self.ctx.publish(T, rows=np.ascontiguousarray(self.packed[r])) for r in range(R)]
        assert ids == list(range(R))
        self.req = [int(r) for r in order]
        self.req_dev = torch.tensor(self.req, dtype=torch.int32, device="cuda")
        self.topk = np.stack([np.stack([rng.permutation(T)[:k] for _ in range(L)]) for _ in range(B)]).astype(np.int32)
        for _ in range(pad):
            self.topk[rng.integers(B), rng.integers(L), rng.integers(k)] = -1
        self.assemble(self.topk)
        self.q = (rng.standard_normal((B * L, 128, 576)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        self.q_dev = _bf16(self.q)

    def assemble(self, topk):
        t = torch.from_numpy(topk).cuda()
        self.slots = torch.empty_like(t)
        n = torch.empty((2, self.B, self.L), dtype=torch.int32, device="cuda")
        self.ctx.assemble(self.req_dev, t, self.slots, n[0], n[1])

    def check(self, out, lse, scale, layer=-1, skip=()):
        units = [(b, l) for b in range(self.B) for l in (range(self.L) if layer < 0 else [layer])]
        out = out.view(torch.int16).cpu().numpy().view(np.uint16)
        lse = lse.cpu().numpy()
        for n, (b, l) in enumerate(units):
            if b in skip:
                assert not out[n].any() and np.all(np.isneginf(lse[n]))
                continue
            tok = self.topk[b, l]
            valid = tok >= 0
            keys = np.zeros((self.k, 576))
            keys[valid] = q4.values(self.packed[self.req[b], l][tok[valid]])
            q = _f64(self.q[n if layer < 0 else n])
            want, want_lse = att.attend(q, keys, valid, scale)
            lse_tol, atol, rtol = ac.bounds(q, keys, valid, scale)
            got = _f64(out[n])
            assert np.all(np.abs(got - want) <= atol + (rtol + ac.MISC) * np.abs(want)), (b, l, np.abs(got - want).max())
            both = np.isneginf(want_lse) & np.isneginf(lse[n])
            with np.errstate(invalid="ignore"):
                d = np.where(both, 0.0, np.abs(lse[n] - want_lse))
            assert np.all(d <= lse_tol + ac.MISC), (b, l, d.max())


def _outputs(units):
    return (torch.full((units, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda"),
            torch.full((units, 128), float("nan"), device="cuda"))


@pytest.mark.parametrize("k,T", [(1, 1), (1, 5), (20, 64), (63, 100), (64, 100), (65, 100), (129, 200), (300, 400),
                                 (1000, 1024), (2048, 2100), (4096, 4200)])
def test_attention_of_one_unit_at_block_borders(k, T):
    """One unit: its keys are split over every SM pair there is."""
    c = Cache(1, 1, T, k, seed=k)
    out, lse = _outputs(1)
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, out, lse, sm_scale=1 / 24)
    c.check(out, lse, 1 / 24)
    assert c.ctx.get_device_error() == 0
    c.ctx.close()


@pytest.mark.parametrize("B,L,k,sms,scale", [(3, 2, 300, 0, 1 / 24), (3, 2, 300, 0, 0.3), (3, 2, 300, 4, 0.3), (3, 2, 300, 2, 0.3),
                                             (5, 3, 130, 0, 0.1), (20, 4, 70, 0, 0.1), (26, 3, 200, 0, 0.1), (7, 1, 511, 40, 0.1)])
def test_attention_splits_and_waves(B, L, k, sms, scale):
    """Units fewer than, equal to and more than the SM pairs; pads among the keys; a request order of its own."""
    c = Cache(B, L, k + 50, k, seed=B, pad=40, R=B + 1)
    out, lse = _outputs(B * L)
    c.ctx.set_attend_sms(sms)
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, out, lse, sm_scale=scale)
    c.check(out, lse, scale)
    assert c.ctx.get_device_error() == 0
    c.ctx.close()


@pytest.mark.parametrize("sms", [0, 2])
def test_attention_of_empty_units_and_non_requests(sms):
    """A unit that selects nothing, one whose keys fill only its last block, and an entry that is no request (split
    over several SM pairs, and not)."""
    c = Cache(4, 1, 400, 320, seed=9)
    c.topk[1] = -1
    c.topk[2, 0, :318] = -1
    c.assemble(c.topk)
    req = c.req_dev.clone()
    req[3] = 77
    out, lse = _outputs(4)
    c.ctx.set_attend_sms(sms)
    c.ctx.attend_q4(req, c.q_dev, c.slots, out, lse, sm_scale=0.2)
    c.check(out, lse, 0.2, skip=(3,))
    assert not out[1].any() and bool(torch.isneginf(lse[1]).all())
    c.ctx.close()


def test_attention_of_one_layer_without_lse_and_in_a_graph():
    c = Cache(3, 3, 300, 200, seed=11, pad=5)
    layer = 2
    q = c.q_dev.view(3, 3, 128, 576)[:, layer].contiguous()
    c.q = c.q.reshape(3, 3, 128, 576)[:, layer].copy()
    slots = c.slots[:, layer].contiguous()
    out, lse = _outputs(3)
    c.ctx.attend_q4(c.req_dev, q, slots, out, lse, layer=layer, sm_scale=0.1)
    c.check(out, lse, 0.1, layer=layer)
    alone = torch.empty_like(out)
    c.ctx.attend_q4(c.req_dev, q, slots, alone, layer=layer, sm_scale=0.1)
    assert torch.equal(alone.view(torch.int16), out.view(torch.int16))
    g = torch.cuda.CUDAGraph()
    replayed = torch.empty_like(out)
    with torch.cuda.graph(g):
        c.ctx.attend_q4(c.req_dev, q, slots, replayed, layer=layer, sm_scale=0.1)
    for _ in range(3):
        replayed.zero_()
        g.replay()
        assert torch.equal(replayed.view(torch.int16), out.view(torch.int16))  # the same bits every time
    c.ctx.close()


def test_masked_rows_and_rows_behind_the_selection_are_not_read():
    """Rows that no slot names may hold anything: NaN scales and codes there change nothing."""
    c = Cache(2, 1, 600, 128, seed=13, S=500)
    c.topk[:, :, 100:] = -1
    c.assemble(c.topk)
    out, lse = _outputs(2)
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, out, lse, sm_scale=0.1)
    c.check(out, lse, 0.1)
    base, stride = c.ctx.hot_buffer()
    assert stride == 500 * ROW

    class Mem:
        __cuda_array_interface__ = {"shape": (2, 500, ROW), "typestr": "|u1", "data": (base, False), "version": 3}
    hot = torch.as_tensor(Mem(), device="cuda")
    for b in range(2):
        used = torch.zeros(500, dtype=torch.bool, device="cuda")
        s = c.slots[b, 0]
        used[s[s >= 0].long()] = True
        hot[c.req[b]][~used] = 0xFF
    again, lse2 = _outputs(2)
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, again, lse2, sm_scale=0.1)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse, lse2)
    c.ctx.close()


@pytest.mark.parametrize("k", [64, 256])
def test_attention_equals_skv_attend_over_the_unpacked_rows(k):
    """The same values as bf16 rows in another context, one block of keys and several: the score dims are split
    between the two CTAs in another way, the partial scores cross with more bits and the references are raised at different thresholds, so each of skv_attend and
    skv_attend_q4 is within the derived bounds of the same value."""
    c = Cache(80, 1, 300, k, seed=17)
    rows = torch.empty((80 * 300, 576), dtype=torch.bfloat16, device="cuda")
    c.ctx.unpack_rows(torch.from_numpy(c.packed.reshape(-1, ROW)).cuda(), rows)
    with _ctx(80, 1, 300, k, k, 80, row_bytes=1152) as wide:
        for r in range(80):
            wide.publish(300, rows=rows[300 * r:300 * (r + 1)])
        slots = torch.empty_like(c.slots)
        n = torch.empty((2, 80, 1), dtype=torch.int32, device="cuda")
        wide.assemble(c.req_dev, torch.from_numpy(c.topk).cuda(), slots, n[0], n[1])
        assert torch.equal(slots, c.slots)
        a, la = _outputs(80)
        b, lb = _outputs(80)
        wide.attend(c.req_dev, c.q_dev, slots, a, la, sm_scale=0.2)
        c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, b, lb, sm_scale=0.2)
        c.check(a, la, 0.2)
        c.check(b, lb, 0.2)
    c.ctx.close()


@pytest.mark.parametrize("k,sms", [(64, 2), (300, 2), (300, 0)])
def test_scores_of_twenty_bits_are_exact(k, sms):
    """Codes under the scale 1 and whole q up to 127: a partial score is a multiple of 1/2 and at most 288 * 6 * 127 <
    2^18, so of at most 19 bits; it is summed exactly in fp32 and crosses the pair as fp32.  What is left on lse: the
    scale's and the maximum's roundings (2^-24 of the largest scaled score each, and its log2 form's), MISC, and the
    fp32 sum; the 24 bits of skv_attend would be off by 2^-17 of a partial score, ten times that."""
    c = Cache(2, 1, 400, k, seed=29)
    rng = np.random.default_rng(29)
    c.packed[..., :288] = rng.integers(0, 256, c.packed[..., :288].shape)
    c.packed[..., 288:324] = 0x38
    c.packed[..., 324] = 127
    for r in range(2):
        c.ctx.release(r)
    ids = [c.ctx.publish(400, rows=np.ascontiguousarray(c.packed[r])) for r in range(2)]
    c.packed = c.packed[np.argsort(ids)]
    c.assemble(c.topk)
    q = rng.integers(-127, 128, (2, 128, 576)).astype(np.float32)
    c.q = (q.view(np.uint32) >> 16).astype(np.uint16)
    assert np.array_equal(_f64(c.q), q)
    scale = 2.0 ** -9
    out, lse = _outputs(2)
    c.ctx.set_attend_sms(sms)
    c.ctx.attend_q4(c.req_dev, _bf16(c.q), c.slots, out, lse, sm_scale=scale)
    c.check(out, lse, scale)
    lse = lse.cpu().numpy()
    for b in range(2):
        keys = q4.values(c.packed[c.req[b], 0][c.topk[b, 0]])
        x = _f64(c.q[b]) @ keys.T * scale
        _, want = att.attend(_f64(c.q[b]), keys, np.ones(k, bool), scale)
        tol = 2 * ac.MISC + (k / 32 + 64) * 2.0 ** -24 + 4 * 2.0 ** -24 * np.abs(x).max(axis=1)
        assert np.all(np.abs(lse[b] - want) <= tol), (np.abs(lse[b] - want).max(), tol.max())
    c.ctx.close()


@pytest.mark.parametrize("sms", [0, 2])
@pytest.mark.parametrize("k,at,group", [(1, 0, 0), (1, 0, 35), (200, 5, 0), (200, 40, 0), (200, 5, 35), (200, 199, 35), (200, 130, 17)])
def test_a_key_that_is_nan_makes_its_unit_nan(k, at, group, sms):
    """A NaN group gives every head a NaN score (in either half of the dims and of a block's keys, alone or not)."""
    c = Cache(3, 1, 300, k, seed=31)
    base, stride = c.ctx.hot_buffer()

    class Mem:
        __cuda_array_interface__ = {"shape": (3, k, ROW), "typestr": "|u1", "data": (base, False), "version": 3}
    assert stride == k * ROW
    torch.as_tensor(Mem(), device="cuda")[c.req[1], int(c.slots[1, 0, at]), 288 + group] = 0x7F
    out, lse = _outputs(3)
    out.zero_()
    lse.zero_()
    c.ctx.set_attend_sms(sms)
    c.ctx.attend_q4(c.req_dev, c.q_dev, c.slots, out, lse, sm_scale=0.1)
    assert bool(torch.isnan(out[1].float()).all()) and bool(torch.isnan(lse[1]).all())
    keep = torch.tensor([0, 2], device="cuda")
    c.B, c.req, c.topk, c.q = 2, [c.req[0], c.req[2]], c.topk[[0, 2]], c.q[[0, 2]]
    c.check(out[keep], lse[keep], 0.1)
    assert c.ctx.get_device_error() == 0
    c.ctx.close()


def test_attention_refuses_bad_arguments():
    c = Cache(2, 2, 50, 16, seed=19)
    out, lse = _outputs(4)
    bad = skv.SKV_ERR_INVALID_ARG
    args = (c.req_dev.data_ptr(), 2, -1, c.q_dev.data_ptr(), c.slots.data_ptr(), out.data_ptr(), lse.data_ptr(), 0.1, 0)
    for at, v in ((0, 0), (1, -1), (1, 3), (2, 2), (2, -2), (3, 0), (3, args[3] + 2), (4, 0), (5, 0), (5, args[5] + 8),
                  (7, 0.0), (7, -1.0), (7, float("nan")), (7, float("inf"))):
        a = list(args)
        a[at] = v
        assert skv.skv_attend_q4(c.ctx.h, *a) == bad, (at, v)
    assert skv.skv_attend_q4(None, *args) == bad
    assert skv.skv_attend(c.ctx.h, *args) == bad  # packed rows are not bf16 rows
    with _ctx(2, 2, 50, 16, 16, 2, row_bytes=1152) as wide:
        assert skv.skv_attend_q4(wide.h, *args) == bad
    torch.cuda.synchronize()
    assert bool(torch.isnan(out.float()).all()) and SKV_Q4_ROW_BYTES == ROW
    c.ctx.close()
