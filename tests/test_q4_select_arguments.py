"""The Python side of the calls around a cache in 4 bits refuses tensors of another
type, size or place before anything reaches the library (no GPU: the context here
has no handle, which the library would refuse with another error)."""
import pytest
import torch

from sparse_attention_kv_skv_gb300 import build

build.build()

from sparse_attention_kv_skv_gb300 import Config, Context, Index, SkvError  # noqa: E402
from sparse_attention_kv_skv_gb300 import skv  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture
def ctx(monkeypatch):
    """A context without a handle, for which host memory is the device's (unless a test asks otherwise)."""
    c = Context.__new__(Context)
    c.cfg = Config(max_requests=2, num_layers=3, max_context=40, topk=8, hot_slots=8, max_batch=2, row_bytes=336, device=-1)
    c.h = None
    monkeypatch.setattr(skv, "_raw_stream", lambda device: 0)
    return c


def _pack(ctx, rows=BF16, packed=torch.uint8, values=BF16, n=4):
    ctx.pack_rows(torch.zeros((n, 576), dtype=rows), torch.zeros((4, 336), dtype=packed), torch.zeros((4, 576), dtype=values))


def _unpack(ctx, values=BF16, n=4):
    ctx.unpack_rows(torch.zeros((4, 336), dtype=torch.uint8), torch.zeros((n, 576), dtype=values))


def _select(ctx, q=BF16, w=torch.float32, topk=torch.int32, req=torch.int32, work=1 << 20, keys=BF16, B=2, layer=-1):
    units = B if layer >= 0 else 3 * B
    index = Index(torch.zeros((2, 3, 40, 64), dtype=keys))
    ctx.select(index, torch.zeros(2, dtype=req), torch.zeros((units, 4, 64), dtype=q), torch.zeros((units, 4), dtype=w),
               torch.zeros((units, 8), dtype=topk), torch.zeros(work, dtype=torch.uint8), layer=layer, B=B)


def _attend(ctx, req=torch.int32, q=BF16, slots=torch.int32, out=BF16, lse=torch.float32, units=6, layer=-1):
    ctx.attend_q4(torch.zeros(2, dtype=req), torch.zeros((units, 128, 576), dtype=q), torch.zeros((units, 8), dtype=slots),
                  torch.zeros((units, 128, 512), dtype=out), None if lse is None else torch.zeros((units, 128), dtype=lse),
                  layer=layer)


@pytest.mark.parametrize("call,good", [
    (_pack, {}), (_pack, dict(packed=torch.int8)), (_unpack, {}), (_select, {}), (_select, dict(layer=1)), (_select, dict(B=1)),
    (_attend, {}), (_attend, dict(lse=None)), (_attend, dict(layer=2, units=2)), (_attend, dict(units=7))])
def test_the_right_arguments_reach_the_library(ctx, call, good):
    with pytest.raises(SkvError):  # no handle
        call(ctx, **good)


@pytest.mark.parametrize("call,bad", [
    (_pack, dict(rows=torch.float16)), (_pack, dict(rows=torch.int16)), (_pack, dict(rows=torch.float32)),
    (_pack, dict(values=torch.float16)), (_pack, dict(values=torch.float32)), (_pack, dict(n=5)),
    (_unpack, dict(values=torch.float16)), (_unpack, dict(values=torch.float32)), (_unpack, dict(n=3)),
    (_select, dict(keys=torch.float16)), (_select, dict(q=torch.float16)), (_select, dict(q=torch.float32)),
    (_select, dict(w=torch.float64)), (_select, dict(w=BF16)), (_select, dict(topk=torch.int64)), (_select, dict(topk=torch.float32)),
    (_select, dict(req=torch.int64)),
    (_attend, dict(q=torch.float16)), (_attend, dict(q=torch.float32)), (_attend, dict(slots=torch.int64)),
    (_attend, dict(out=torch.float32)), (_attend, dict(out=torch.float16)), (_attend, dict(lse=torch.float64)),
    (_attend, dict(lse=BF16)), (_attend, dict(req=torch.int64)), (_attend, dict(units=5))])
def test_other_types_and_sizes_are_refused(ctx, call, bad):
    with pytest.raises(ValueError):
        call(ctx, **bad)


@pytest.mark.parametrize("call", [_pack, _unpack, _select, _attend])
def test_tensors_elsewhere_than_the_contexts_device_are_refused(ctx, call):
    ctx.cfg.device = 0  # host memory that is not pinned is not the device's
    with pytest.raises(ValueError, match="device"):
        call(ctx)


def test_tensors_that_are_not_contiguous_are_refused(ctx):
    q = torch.zeros((6, 128, 2 * 576), dtype=BF16)[..., ::2]
    slots, out = torch.zeros((6, 8), dtype=torch.int32), torch.zeros((6, 128, 512), dtype=BF16)
    with pytest.raises(ValueError, match="contiguous"):
        ctx.attend_q4(torch.zeros(2, dtype=torch.int32), q, slots, out)


def test_an_index_that_is_changed_after_a_call_is_described_anew():
    keys = torch.zeros((2, 3, 40, 64), dtype=BF16)
    index = Index(keys, block=2, first=1, last=1)
    before = index.c(4)._obj
    index.block, index.first, index.last, index.relu = 4, 0, 2, False
    index.keys = torch.zeros((2, 3, 20, 128), dtype=BF16)
    s = index.c(4)._obj
    assert (s.block, s.first, s.last, s.relu, s.dim, s.key_stride) == (4, 0, 2, 0, 128, 256)
    assert s.keys == index.keys.data_ptr() and (before.block, before.dim) == (2, 64)  # a call under way keeps its own
    with pytest.raises(ValueError):
        index.keys = keys.half()
