"""The Python side of the calls around a shared prefix refuses tensors of another
type, size, order or place before anything reaches the library (no GPU: the context
here has no handle, which the library would refuse with another error)."""
import pytest
import torch

from sparse_attention_kv_skv_gb300 import build

build.build()

from sparse_attention_kv_skv_gb300 import Config, Context, Prefix, SkvError  # noqa: E402
from sparse_attention_kv_skv_gb300 import skv  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
L, N, H = 3, 40, 16


@pytest.fixture
def ctx(monkeypatch):
    """A context without a handle, for which host memory is the device's (unless a test asks otherwise)."""
    c = Context.__new__(Context)
    c.cfg = Config(max_requests=1, num_layers=L, max_context=1, topk=1, hot_slots=1, max_batch=4, device=-1)
    c.h = None
    monkeypatch.setattr(skv, "_raw_stream", lambda device: 0)
    return c


def _prefix(layers=L, n=N):
    return Prefix(torch.zeros((layers, n, 576), dtype=BF16))


def _attend(ctx, layers=L, q=BF16, out=BF16, lse=F32, units=6, of=6, dim=576, layer=-1, B=None, work=64):
    ctx.attend_prefix(_prefix(layers), torch.zeros((units, H, dim), dtype=q), torch.zeros((of, H, 512), dtype=out),
                      None if lse is None else torch.zeros((of, H), dtype=lse), torch.zeros(work, dtype=torch.uint8), layer=layer, B=B)


def _weigh(ctx, layers=L, q=BF16, lse=F32, weights=F32, out=F32, units=6, w=(L, N), o=(L, N), layer=-1, lses=6):
    ctx.weigh_prefix(_prefix(layers), torch.zeros((units, H, 576), dtype=q), torch.zeros((lses, H), dtype=lse),
                     None if weights is None else torch.zeros(w, dtype=weights), torch.zeros(o, dtype=out),
                     torch.zeros(64, dtype=torch.uint8), layer=layer)


def _evict(ctx, layers=L, weights=F32, w=(L, N), kept=torch.int32, rows=BF16, kw=F32, of=L, layer=-1):
    ctx.evict_prefix(_prefix(layers), torch.zeros(w, dtype=weights), torch.zeros((of, 8), dtype=kept),
                     None if rows is None else torch.zeros((of, 8, 576), dtype=rows),
                     None if kw is None else torch.zeros((of, 8), dtype=kw), torch.zeros(64, dtype=torch.uint8), layer=layer)


def _join(ctx, parts=2, o=BF16, e=F32, out=BF16, lse=F32, n=5, of=5, width=512, lses=None):
    ctx.join([torch.zeros((n, width), dtype=o)] * parts, [torch.zeros(n, dtype=e)] * (parts if lses is None else lses),
             torch.zeros((of, width), dtype=out), None if lse is None else torch.zeros(of, dtype=lse))


@pytest.mark.parametrize("call,good", [
    (_attend, {}), (_attend, dict(lse=None)), (_attend, dict(layer=1, units=2, of=2)), (_attend, dict(B=1)), (_attend, dict(of=7)),
    (_attend, dict(layers=L + 1)), (_weigh, {}), (_weigh, dict(weights=None)), (_weigh, dict(o=(L, N + 3))), (_weigh, dict(layer=2, units=2)),
    (_evict, {}), (_evict, dict(rows=None)), (_evict, dict(kw=None)), (_evict, dict(layer=0, of=1)), (_evict, dict(w=(L + 1, N + 5))),
    (_join, {}), (_join, dict(lse=None)), (_join, dict(parts=8)), (_join, dict(parts=1))])
def test_the_right_arguments_reach_the_library(ctx, call, good):
    with pytest.raises(SkvError):  # no handle
        call(ctx, **good)


@pytest.mark.parametrize("call,bad", [
    (_attend, dict(q=torch.float16)), (_attend, dict(q=F32)), (_attend, dict(out=F32)), (_attend, dict(out=torch.float16)),
    (_attend, dict(lse=BF16)), (_attend, dict(lse=torch.float64)), (_attend, dict(units=5)), (_attend, dict(units=7, of=7)),
    (_attend, dict(of=5)), (_attend, dict(dim=512)), (_attend, dict(B=3)), (_attend, dict(layers=L - 1)),
    (_weigh, dict(q=F32)), (_weigh, dict(lse=torch.float64)), (_weigh, dict(lses=5)), (_weigh, dict(weights=torch.float64)),
    (_weigh, dict(out=BF16)), (_weigh, dict(w=(L, N - 1))), (_weigh, dict(o=(L, N - 1))), (_weigh, dict(o=(L - 1, N))),
    (_weigh, dict(o=(L * N,))), (_weigh, dict(layers=L - 1)), (_weigh, dict(units=4)),
    (_evict, dict(weights=torch.float64)), (_evict, dict(w=(L, N - 1))), (_evict, dict(kept=torch.int64)), (_evict, dict(rows=torch.float16)),
    (_evict, dict(kw=BF16)), (_evict, dict(of=L - 1)), (_evict, dict(layers=L - 1)),
    (_join, dict(parts=0)), (_join, dict(parts=9)), (_join, dict(lses=1)), (_join, dict(o=torch.float16)), (_join, dict(e=torch.float64)),
    (_join, dict(out=F32)), (_join, dict(lse=BF16)), (_join, dict(n=4)), (_join, dict(of=4)), (_join, dict(width=576))])
def test_other_types_and_sizes_are_refused(ctx, call, bad):
    with pytest.raises(ValueError):
        call(ctx, **bad)


@pytest.mark.parametrize("call", [_attend, _weigh, _evict, _join])
def test_tensors_elsewhere_than_the_contexts_device_are_refused(ctx, call):
    ctx.cfg.device = 0
    with pytest.raises(ValueError, match="device"):
        call(ctx)


def test_tensors_of_another_order_are_refused(ctx):
    p, work = _prefix(), torch.zeros(64, dtype=torch.uint8)
    q, out, lse = torch.zeros((6, H, 576), dtype=BF16), torch.zeros((6, H, 512), dtype=BF16), torch.zeros((6, H))
    apart = torch.zeros((6, H, 2 * 576), dtype=BF16)[..., ::2]
    with pytest.raises(ValueError, match="contiguous"):
        ctx.attend_prefix(p, apart, out, lse, work)
    with pytest.raises(ValueError, match="contiguous"):
        ctx.attend_prefix(p, q, torch.zeros((6, 512, H), dtype=BF16).transpose(1, 2), lse, work)
    with pytest.raises(ValueError, match="adjacent"):
        ctx.weigh_prefix(p, q, lse, None, torch.zeros((N, L)).T, work)
    for rows in (torch.zeros((L, N, 576)), torch.zeros((L, N, 640), dtype=BF16), torch.zeros((N, 576), dtype=BF16),
                 torch.zeros((L, N, 2 * 576), dtype=BF16)[..., ::2]):
        with pytest.raises(ValueError):
            Prefix(rows)


def test_a_prefix_that_is_changed_is_described_anew():
    p = _prefix()
    before = p.c()._obj
    p.rows = torch.zeros((L, 2 * N, 640), dtype=BF16)[:, :N + 2, :576]
    s = p.c()._obj
    assert (s.n, s.row_stride, s.layer_stride, p.n) == (N + 2, 1280, 1280 * 2 * N, N + 2)
    assert s.rows == p.rows.data_ptr() and (before.n, before.row_stride) == (N, 1152)  # a call under way keeps its own
    with pytest.raises(ValueError):
        p.rows = p.rows.half()
    assert p.n == N + 2


STREAM_CALLS = {
    "attend_prefix": lambda c, **k: c.attend_prefix(_prefix(), torch.zeros((L, H, 576), dtype=BF16), torch.zeros((L, H, 512), dtype=BF16), None,
                                                    torch.zeros(64, dtype=torch.uint8), **k),
    "join": lambda c, **k: c.join([torch.zeros((1, 512), dtype=BF16)], [torch.zeros(1)], torch.zeros((1, 512), dtype=BF16), **k),
    "weigh_prefix": lambda c, **k: c.weigh_prefix(_prefix(), torch.zeros((L, H, 576), dtype=BF16), torch.zeros((L, H)), None,
                                                  torch.zeros((L, N)), torch.zeros(64, dtype=torch.uint8), **k),
    "evict_prefix": lambda c, **k: c.evict_prefix(_prefix(), torch.zeros((L, N)), torch.zeros((L, 4), dtype=torch.int32), None, None,
                                                  torch.zeros(64, dtype=torch.uint8), **k),
    "selftest_prefix_timeout": lambda c, **k: c.selftest_prefix_timeout(_prefix(), torch.zeros((L, H, 576), dtype=BF16), None,
                                                                        torch.zeros((L, H, 512), dtype=BF16), None,
                                                                        torch.zeros(64, dtype=torch.uint8), **k),
}


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_a_call_goes_to_the_stream_given_or_to_the_devices_current_one(ctx, monkeypatch, name):
    asked = []
    monkeypatch.setattr(skv, "_raw_stream", lambda device: asked.append(device) or 0)
    with pytest.raises(SkvError):
        STREAM_CALLS[name](ctx)
    assert asked == [-1]
    with pytest.raises(SkvError):
        STREAM_CALLS[name](ctx, stream=0)
    assert asked == [-1]


def test_every_call_around_a_prefix_that_takes_a_stream_is_covered():
    import inspect
    takes = {n for n, f in vars(skv.PrefixCalls).items() if callable(f) and "stream" in inspect.signature(f).parameters}
    assert takes == set(STREAM_CALLS)
