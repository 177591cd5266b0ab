"""A context of packed rows has an allocation more than others, the scratch of split
units; here it fails (a host-side fake of the failing call)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_kv_skv_gb300 import Config, Context, SkvError, skv


def test_scratch_that_cannot_be_allocated_fails_the_create(monkeypatch):
    """The 18th allocation of a context of packed rows: SKV_ERR_OOM, nothing is left behind, a later create succeeds."""
    cfg = Config(max_requests=4, num_layers=2, max_context=4096, topk=256, hot_slots=512, max_batch=4, row_bytes=336)
    monkeypatch.delenv("SKV_TEST_FAIL_ALLOC", raising=False)
    Context(cfg).close()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        monkeypatch.setenv("SKV_TEST_FAIL_ALLOC", "18")
        with pytest.raises(SkvError) as e:
            Context(cfg)
        assert e.value.status == skv.SKV_ERR_OOM
        assert b"out of memory" in skv.skv_last_cuda_error()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    monkeypatch.setenv("SKV_TEST_FAIL_ALLOC", "19")  # past the last allocation: nothing fails
    with Context(cfg) as ctx:
        assert ctx.publish(100) == 0
    monkeypatch.delenv("SKV_TEST_FAIL_ALLOC")
