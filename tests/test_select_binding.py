"""The Python side of skv_select: what an Index hands to the C call (no GPU)."""
import pytest
import torch

from sparse_attention_kv_skv_gb300 import build

build.build()

from sparse_attention_kv_skv_gb300 import Config, Index  # noqa: E402


def test_an_index_used_with_two_head_counts_at_once_keeps_both():
    index = Index(torch.zeros((2, 3, 40, 64), dtype=torch.bfloat16), block=2, first=1, last=1, relu=False)
    a, b = index.c(4)._obj, index.c(16)._obj
    assert (a.heads, b.heads) == (4, 16) and index.c(4)._obj is a
    for s in (a, b):
        assert (s.dim, s.block, s.first, s.last, s.relu) == (64, 2, 1, 1, 0)
        assert (s.request_stride, s.layer_stride, s.key_stride) == (3 * 40 * 128, 40 * 128, 128)
        assert s.keys == index.keys.data_ptr()


def test_an_index_refuses_keys_that_are_not_adjacent_bf16_rows():
    keys = torch.zeros((2, 3, 40, 128), dtype=torch.bfloat16)
    for bad in (keys[0], keys[..., ::2], keys.float(), keys.view(torch.int16)):
        with pytest.raises(ValueError):
            Index(bad)


def test_an_index_fits_a_context_by_requests_layers_and_tokens():
    index = Index(torch.zeros((2, 3, 40, 64), dtype=torch.bfloat16), block=4)
    cfg = dict(max_requests=2, num_layers=3, max_context=160, topk=8, hot_slots=8, max_batch=1)
    assert index.fits(Config(**cfg))
    for name in ("max_requests", "num_layers", "max_context"):
        assert not index.fits(Config(**{**cfg, name: cfg[name] + 1}))
