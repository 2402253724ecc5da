"""Handles of emb_create_history in the binding's calls (CPU): they are known without a HistoryAttention, and those that
are not, or no longer, are refused as such."""
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_history_abi import cache, handle


def calls(h, kv):
    q, k = torch.zeros((3, 8, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i, lse, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 8), torch.zeros(16, dtype=torch.uint8)
    return [lambda: E.emb_history_attention(h, q, k, k, q, i),
            lambda: E.emb_history_attention_backward(h, q, k, k, q, lse, q, q, k, k, i, ws),
            lambda: E.emb_history_step(h, kv, q, q, i, torch.zeros((3, 1), dtype=torch.int32), ws)]


def test_a_created_handle_is_known():
    h, kv = handle(), cache()
    for call in calls(h, kv):
        with pytest.raises(ValueError, match="not in device memory"):       # past the handle, up to the operands
            call()
    wrong = torch.zeros((3, 7, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        E.emb_history_step(h, kv, wrong, wrong, None, None, None)
    E.emb_destroy_history(h)
    for call in calls(h, kv):
        with pytest.raises(ValueError, match="not a handle"):
            call()
    E.emb_destroy_kv(kv)


def test_no_handle():
    for call in calls(None, None):
        with pytest.raises(ValueError, match="not a handle"):
            call()


@pytest.mark.parametrize("kw,want", [
    (dict(), (8, 2, 64, torch.bfloat16, 32)), (dict(t=E.EMB_F16, causal=0, dim=96), (8, 2, 96, torch.float16, 64)),
    (dict(buckets=0, exact=0, far=0, causal=0), (8, 2, 64, torch.bfloat16, 0))])
def test_what_a_handle_stands_for(kw, want):
    h = handle(**kw)
    assert E._history(h) == want
    E.emb_destroy_history(h)
    assert h not in E._histories
