"""GPU test of candidate ranking over users' histories (dlrm_sparse_embedding_amd/ranking.py): embedding
rows, projection, per-head norm or rotation, append, attention and a training step together, against the
64-bit definitions of the sequence operators. Tolerances as in test_gpu_sequence.py: u = 2^-24, h = 2^-8
(half a bf16 step); what the cache holds is read back from it, so each step's own rounding counts alone."""
import math

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd.ranking import HistoryRanker
from oracle import sequence_oracle as S

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8


def n64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("norm,layout", [(True, "half"), (False, "interleaved")])
def test_rank_and_train(norm, layout):
    gen = torch.Generator().manual_seed(3)
    lens, counts = [70, 0, 33], [5, 2, 9]
    r = HistoryRanker(500, width=32, heads=4, kv_heads=2, dim=64, pages=64, norm=norm, layout=layout)
    if norm:
        r.wq.mul_((1 + 0.2 * torch.randn(64, generator=gen)).cuda())
        r.wk.mul_((1 + 0.2 * torch.randn(64, generator=gen)).cuda())
    history = torch.randint(0, 500, (sum(lens),), generator=gen).cuda()
    ids = torch.randint(0, 500, (sum(counts),), generator=gen).cuda()
    table, own = r.new_pages(lens), r.new_pages([1] * len(ids))
    offsets = i32(np.concatenate([[0], np.cumsum(lens)]))
    groups = np.concatenate([[0], np.cumsum(counts)])
    r.append(history, offsets, i32(lens), table)
    out, lse = r.rank(ids, i32(groups), i32(lens), table, own)
    r.cache.check_error()
    r.tables.check_device_error()

    spec = dict(rot=64, layout=layout)
    w = lambda t: n64(t) if norm else None
    placed = lambda x, pos, wt: S.norm_rotary(x, pos, wt, 1e-6, **spec) if norm else S.rotate(x, pos, **spec)
    # keys as written: one bf16 rounding of the definition's
    fused = r.project(r.rows(history))
    _, k, v = r.parts(fused)
    pos = np.concatenate([np.arange(n) for n in lens])
    want = placed(n64(k), pos, w(r.wk))
    where = [(int(table[u, s // 16]), s % 16) for u, n in enumerate(lens) for s in range(n)]
    pg, sl = (torch.tensor(x).cuda() for x in zip(*where))
    top = np.abs(want).max(-1, keepdims=True)
    assert (np.abs(n64(r.cache.k[pg, sl]) - want) <= H * 1.001 * np.abs(want) + 64 * U * top).all()
    assert torch.equal(r.cache.v[pg, sl], v)
    # the attention over what the cache holds
    q, kc, _ = r.parts(r.project(r.rows(ids)))
    place = np.repeat(lens, counts)
    qr, _ = r.place(q, None, torch.tensor(place).cuda())
    o, z, bound = S.prefix_attention(n64(qr), n64(r.cache.k), n64(r.cache.v), 1 / math.sqrt(64), np.arange(len(ids) + 1),
                                     [1] * len(ids), own.cpu().numpy(), groups, lens, table.cpu().numpy())
    kmax = np.repeat(np.abs(n64(r.cache.k)).max((0, 1)), 2, 0)
    e = (64 + 8) * U / math.sqrt(64) * (np.abs(n64(qr)) * kmax).sum(-1)
    assert (np.abs(n64(out) - o) <= (H + 2 * e[..., None] + 128 * U) * bound + H * 1.001 * np.abs(o) + 1e-38).all()
    assert (np.abs(n64(lse) - z) <= e + 256 * U + 4 * U * np.abs(z)).all()

    # gradients of the placed queries and keys
    dq, dk = (torch.randn((len(ids), n, 64), generator=gen).bfloat16().cuda() for n in (4, 2))
    gq, gk, dwq, dwk = r.place_backward(q, kc, torch.tensor(place).cuda(), dq, dk)
    for x, dy, g, wt, dw in ((q, dq, gq, r.wq, dwq), (kc, dk, gk, r.wk, dwk)):
        if norm:
            want, want_w = S.norm_rotary_grad(n64(x), n64(dy), place, n64(wt), 1e-6, **spec)
            inv = 1 / np.sqrt((n64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
            size = np.abs(n64(wt)).max() * 2 * np.abs(n64(dy)).max(-1, keepdims=True)
            nrm = np.abs(n64(x) * inv)
            err = 40 * U * inv * size * (1 + nrm * nrm.mean(-1, keepdims=True))
            bound_w = (2 * np.abs(n64(dy)).max(-1, keepdims=True) * nrm).sum((0, 1))
            assert (np.abs(n64(dw) - want_w) <= 100 * U * bound_w + U * np.abs(want_w)).all()
        else:
            want = S.rotate(n64(dy), place, inverse=True, **spec)
            err = 16 * U * np.abs(n64(dy)).max(-1, keepdims=True)
        assert (np.abs(n64(g) - want) <= err + H * 1.001 * np.abs(want)).all()

    # a step moves the rows of the items it saw, and no others
    before = r.tables.weights[0][0].clone()
    r.train_step(ids, torch.tensor(place).cuda(), dq, dk, torch.zeros_like(dk), lr=0.05)
    r.tables.check_device_error()
    moved = (r.tables.weights[0][0] != before).any(1).nonzero().flatten()
    assert torch.equal(moved, torch.unique(ids))
    r.close()


def test_no_pages_left():
    r = HistoryRanker(50, width=32, pages=4)
    r.new_pages([16, 17])
    with pytest.raises(ValueError, match="no pages left"):
        r.new_pages([17])
    r.close()
