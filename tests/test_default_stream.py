"""Without a stream argument every call of a context goes to the current stream of
the context's device, whatever device is current, so that calls on one context are
ordered.  (No GPU: the context has no handle, which the library refuses, and the
stream look-up is a stand-in that notes the device it was asked for.)"""
import numpy as np
import pytest
import torch

from sparse_attention_kv_skv_gb300 import build

build.build()

from sparse_attention_kv_skv_gb300 import Config, Context, Index, SkvError  # noqa: E402
from sparse_attention_kv_skv_gb300 import skv  # noqa: E402

I = torch.zeros(64, dtype=torch.int32)

CALLS = {
    "publish": lambda c, **k: c.publish(1, **k),
    "release": lambda c, **k: c.release(0, **k),
    "write_back": lambda c, **k: c.write_back(I[:1], I, **k),
    "extend": lambda c, **k: c.extend(0, I, 1, **k),
    "assemble": lambda c, **k: c.assemble(I[:1], I, I, I, I, **k),
    "assemble_layer": lambda c, **k: c.assemble_layer(0, I[:1], I, I, I, I, **k),
    "assemble_noalloc": lambda c, **k: c.assemble_noalloc(I[:1], I, I, I, I, **k),
    "assemble_host": lambda c, **k: c.assemble_host(*[np.zeros(1, np.int32)] * 5, **k),
    "prefetch": lambda c, **k: c.prefetch(I[:1], I, **k),
    "prefetch_recent": lambda c, **k: c.prefetch_recent(I[:1], 1, **k),
    "attend": lambda c, **k: c.attend(I[:1], I, I, I, **k),
    "attend_q4": lambda c, **k: c.attend_q4(1, 16, 16, 16, B=1, **k),
    "select": lambda c, **k: c.select(Index(torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16)), I[:1],
                                      torch.zeros((1, 1, 64), dtype=torch.bfloat16), torch.zeros((1, 1)), I, I, **k),
    "pack_rows": lambda c, **k: c.pack_rows(torch.zeros((1, 576), dtype=torch.bfloat16), torch.zeros(336, dtype=torch.uint8), **k),
    "unpack_rows": lambda c, **k: c.unpack_rows(torch.zeros(336, dtype=torch.uint8), torch.zeros(576, dtype=torch.bfloat16), **k),
    "selftest_attend_timeout": lambda c, **k: c.selftest_attend_timeout(I[:1], I, I, I, **k),
    "selftest_select_timeout": lambda c, **k: c.selftest_select_timeout(
        Index(torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16)), I[:1], torch.zeros((1, 1, 64), dtype=torch.bfloat16),
        torch.zeros((1, 1)), I, I, **k),
    "get_device_error": lambda c, **k: c.get_device_error(**k),
    "export_state": lambda c, **k: c.export_state(0, **k),
    "export_hot": lambda c, **k: c.export_hot(0, **k),
    "clock": lambda c, **k: c.clock(**k),
    "stats": lambda c, **k: c.stats(**k),
}


@pytest.fixture
def ctx():
    c = Context.__new__(Context)
    # host tensors report the device -1, so the checks of where tensors lie pass
    c.cfg = Config(max_requests=1, num_layers=1, max_context=8, topk=1, hot_slots=1, max_batch=1, device=-1)
    c.h = None
    return c


@pytest.mark.parametrize("name", CALLS)
def test_a_call_without_a_stream_uses_its_devices(ctx, monkeypatch, name):
    asked = []
    monkeypatch.setattr(skv, "_raw_stream", lambda device: asked.append(device) or 0)
    with pytest.raises(SkvError):
        CALLS[name](ctx)
    assert asked == [-1]


@pytest.mark.parametrize("name", CALLS)
def test_a_given_stream_is_used_as_it_is(ctx, monkeypatch, name):
    monkeypatch.setattr(skv, "_raw_stream", lambda device: pytest.fail("the current stream was asked for"))
    with pytest.raises(SkvError):
        CALLS[name](ctx, stream=0)


def test_every_call_that_takes_a_stream_is_covered():
    import inspect
    takes = {n for n, f in vars(Context).items() if callable(f) and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS)
