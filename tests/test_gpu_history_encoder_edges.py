"""GPU tests of the layer over users' histories at its edges: without a bias, and calls without items."""
import pytest
import torch

from dlrm_sparse_embedding_amd.history import HistoryEncoder
from tests.test_gpu_history_encoder import i32, offsets_of

pytestmark = pytest.mark.gpu


def test_no_buckets_is_no_bias():
    a, b = HistoryEncoder(50, buckets=0, pages=8), HistoryEncoder(50, buckets=0, exact=0, far=0, pages=8)
    assert a.bias is None and a.attention.bias_rows == 0
    ids = torch.arange(40, device="cuda")
    for r in (a, b):
        r.y = r.train_step(ids, offsets_of([30, 10]), lambda y: y, 0.1)
    assert torch.equal(a.y, b.y) and torch.equal(a.master, b.master)
    for r in (a, b):
        r.close()


def test_calls_without_items():
    """A step in which nobody has anything changes no weight and no page."""
    r = HistoryEncoder(50, pages=8)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    weights = [r.tables.weights[0][0], r.master, r.proj, r.back_master, r.back, r.norm_w, r.norm_b, r.bias, r.cache.k,
               r.cache.v]
    kept = [w.clone() for w in weights]
    for offsets in (i32([0]), i32([0, 0])):
        assert r.train_step(none, offsets, lambda y: y, 0.1).shape == (0, 128)
    r.append(none, i32([0, 0]), i32([0]), r.new_pages([0]))
    r.append(none, i32([0]), i32([]), r.new_pages([]))
    assert r.step(none, i32([]), r.new_pages([])).shape == (0, 128)
    assert all(torch.equal(x, y) for x, y in zip(kept, weights))
    r.cache.check_error()
    r.attention.check_error()
    r.tables.check_device_error()
    r.close()
