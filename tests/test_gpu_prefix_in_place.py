"""Weights accumulated in place: a layer's new weights may take its old ones' place; rows that overlap otherwise are refused."""
import pytest
import torch

from test_gpu_prefix import Case, _check_weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import SkvError

N = 200


def rows(flat, start, stride, layers=3):
    return flat[start:].as_strided((layers, N), (stride, 1), flat.storage_offset() + start)


@pytest.mark.parametrize("layer", [-1, 0, 1, 2])
@pytest.mark.parametrize("weights,out,refused", [
    ((0, 210), (0, 210), ()),              # in place
    ((0, 210), (0, 230), (-1, 1, 2)),      # the first layer's alone in its place
    ((0, 210), (0, 1000), ()),              # the first layer's in its place, the others apart
    ((0, 210), (8, 210), (-1, 0, 1, 2)),   # a few tokens on
    ((0, 210), (210, 210), (-1,)),         # on the next layer's
    ((0, 420), (210, 420), ()),            # layer by layer side by side
    ((700, 210), (0, 210), ())])
def test_where_new_weights_may_lie(layer, weights, out, refused):
    c = Case(2, 3, N, heads=16)
    lse, flat = c.shares(), torch.rand(3000, device="cuda")
    before, q = flat.clone(), c.q
    w, o = rows(flat, *weights), rows(flat, *out)
    if layer >= 0:
        c.q = q.view(2, 3, 16, 576)[:, layer].contiguous()
    given = lse.view(2, 3, 16)[:, layer].contiguous() if layer >= 0 else lse
    if layer in refused:
        with pytest.raises(SkvError):
            c.weigh(given, w, out=o, layer=layer)
        torch.cuda.synchronize()
        assert torch.equal(flat, before)
    else:
        c.weigh(given, w, out=o, layer=layer)
        c.q = q
        layers = range(3) if layer < 0 else (layer,)
        _check_weights(c, o, lse, rows(before, *weights), layers=layers)
        for l in layers:
            rows(before, *out)[l] = o[l]
        assert torch.equal(flat, before)  # nothing else is written
    assert c.ctx.get_device_error() == 0
