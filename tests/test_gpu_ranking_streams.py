"""GPU tests of ranking on several streams at once: no call's scratch memory is another's."""
import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from dlrm_sparse_embedding_amd.ranking import HistoryRanker

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def ranker(counts, lens):
    gen = torch.Generator().manual_seed(5)
    r = HistoryRanker(500, width=32, heads=4, kv_heads=2, dim=64, pages=700)
    history = torch.randint(0, 500, (sum(lens),), generator=gen).cuda()
    table = r.new_pages(lens)
    r.append(history, i32(np.concatenate([[0], np.cumsum(lens)])), i32(lens), table)
    asked = [(torch.randint(0, 500, (n,), generator=gen).cuda(), i32([0, n // 3, n]), i32(lens), table, r.new_pages([1] * n))
             for n in counts]
    torch.cuda.synchronize()
    return r, asked


def test_each_call_has_its_own_workspace(monkeypatch):
    r, asked = ranker([30, 40], [600, 50])
    taken = []
    # the workspaces alone; nothing is launched on them
    monkeypatch.setattr(E, "emb_prefix_attention", lambda *a, **kw: taken.append(a[10]))
    for args in asked + asked:
        with torch.cuda.stream(torch.cuda.Stream()):
            r.rank(*args)
    torch.cuda.synchronize()
    spans = sorted((w.data_ptr(), w.data_ptr() + w.numel()) for w in taken)
    assert len(spans) == 4 and all(a[1] > a[0] for a in spans)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    r.close()


def test_streams_rank_at_once():
    r, asked = ranker([130, 90, 200], [3000, 50])
    want = [tuple(t.clone() for t in r.rank(*args)) for args in asked]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in asked]
    for _ in range(3):
        got = []
        for st, args in zip(streams, asked):
            with torch.cuda.stream(st):
                got.append(r.rank(*args))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    r.cache.check_error()
    r.close()


def test_calls_without_items():
    # a step in which nobody has anything: no history item, no candidate, no training example
    r, asked = ranker([30], [600, 50])
    want = [t.clone() for t in r.rank(*asked[0])]
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    kept = r.cache.k.clone(), r.cache.v.clone(), r.proj.clone(), r.tables.weights[0][0].clone()
    r.append(none, i32([0, 0]), i32([0]), r.new_pages([0]))
    r.append(none, i32([0]), i32([]), r.new_pages([]))
    out, lse = r.rank(none, i32([0, 0]), i32([600]), asked[0][3][:1].contiguous(), r.new_pages([]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    grads = [torch.empty((0, n, 64), dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2)]
    r.train_step(none, none, *grads, lr=0.1)
    r.cache.check_error()
    r.tables.check_device_error()
    for a, b in zip(kept, (r.cache.k, r.cache.v, r.proj, r.tables.weights[0][0])):
        assert torch.equal(a, b)
    for a, b in zip(want, r.rank(*asked[0])):
        assert torch.equal(a, b)
    r.close()
