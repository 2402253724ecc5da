"""GPU tests of what a training step of the ranker writes: the projection, the norm's weights, the items' rows and
their state, against 64 bits. u = 2^-24, h = 2^-8 (half a bf16 step): a product with the projection's gradients
sums in fp32 and is rounded once, (n + 8) u of the sum of magnitudes and h of the result."""
import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd.ranking import HistoryRanker

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8


def n64(t):
    return t.detach().double().cpu().numpy()


def step_inputs(norm):
    gen = torch.Generator().manual_seed(9)
    r = HistoryRanker(60, width=32, heads=4, kv_heads=2, dim=64, pages=4, norm=norm)
    ids = torch.randint(0, 60, (25,), generator=gen).cuda()         # some items twice
    assert torch.unique(ids).numel() < 25
    place = torch.randint(0, 900, (25,), generator=gen).cuda()
    dq, dk, dv = (torch.randn((25, n, 64), generator=gen).bfloat16().cuda() for n in (4, 2, 2))
    return r, ids, place, dq, dk, dv


def gradients(r, ids, place, dq, dk, dv):
    """(rows as the forward takes them, gradient of the projection's output, of the norm's weights)."""
    rows = r.rows(ids)
    q, k, _ = r.parts(r.project(rows))
    gq, gk, dwq, dwk = r.place_backward(q, k, place, dq, dk)
    return n64(rows.to(r.dtype)), n64(torch.cat([gq, gk, dv], 1)).reshape(25, -1), dwq, dwk


@pytest.mark.parametrize("norm", [True, False])
def test_a_training_step(norm):
    lr, eps = 0.05, 1e-8
    r, ids, place, dq, dk, dv = step_inputs(norm)
    x, g, dwq, dwk = gradients(r, ids, place, dq, dk, dv)
    proj, table = n64(r.proj), n64(r.tables.weights[0][0])
    wq, wk = (r.wq.clone(), r.wk.clone()) if norm else (None, None)
    r.train_step(ids, place, dq, dk, dv, lr=lr)
    r.tables.check_device_error()
    # the projection: its fp32 weights started as what rounds to proj
    dp, size = x.T @ g, np.abs(x).T @ np.abs(g)
    want = proj - lr * dp
    off = lr * ((25 + 8) * U * size + H * np.abs(dp))
    assert (np.abs(n64(r.proj) - want) <= off + H * np.abs(proj) + H * 1.001 * np.abs(want)).all()
    if norm:
        assert torch.equal(r.wq, wq - lr * dwq) and torch.equal(r.wk, wk - lr * dwk)
    # the rows: each lookup's gradient is rounded once, an item's are summed
    d, mag = g @ proj.T, np.abs(g) @ np.abs(proj).T
    err = (g.shape[1] + 8) * U * mag + H * np.abs(d)
    items = ids.cpu().numpy()
    G, e = np.zeros_like(table), np.zeros_like(table)
    for i, item in enumerate(items):
        G[item] += d[i]
        e[item] += err[i]
    e += 32 * U * np.abs(G)
    state = n64(r.tables.state[0][0])
    assert (np.abs(state - G * G) <= 2 * np.abs(G) * e + e * e + 4 * U * G * G).all()
    moved = n64(r.tables.weights[0][0]) - table
    step = np.where(G == 0, 0, -lr * G / (np.abs(G) + eps))
    # a first step's size is the rate; its sign where the gradient is known to that
    tol = np.where(np.abs(G) > 2 * e, lr * (16 * U + 4 * eps / np.maximum(np.abs(G), eps)), 2 * lr) + 2 * U * np.abs(table)
    assert (np.abs(moved - step) <= tol).all()
    assert (np.abs(G) > 2 * e).mean() > 0.3
    rest = np.setdiff1d(np.arange(60), items)
    assert (moved[rest] == 0).all() and (state[rest] == 0).all()
    r.close()


def test_small_steps_are_not_lost():
    # each step moves a weight by at most an eighth of half a bf16 step, 64 of them by several steps
    r, ids, place, dq, dk, dv = step_inputs(True)
    x, g, _, _ = gradients(r, ids, place, dq, dk, dv)
    start = n64(r.proj)
    lr = float(0.3 * H / 8 / np.abs(x.T @ g).max())
    total, off = np.zeros_like(start), np.zeros_like(start)
    for _ in range(64):
        x, g, _, _ = gradients(r, ids, place, dq, dk, dv)
        dp = x.T @ g
        total += lr * dp
        off += lr * ((25 + 8) * U * np.abs(x).T @ np.abs(g) + H * np.abs(dp)) + 2 * U * (np.abs(start) + np.abs(total))
        r.train_step(ids, place, dq, dk, dv, lr=lr)
    want = start - total
    # proj started as the fp32 weights rounded, and is their copy rounded again
    tol = off + H * np.abs(start) + H * 1.001 * np.abs(want)
    big = (np.abs(start) > 0.3) & (np.abs(total) > 2 * tol)
    assert big.any()          # some moved by more than rounding explains
    assert (np.abs(n64(r.proj) - want) <= tol).all()
    r.close()
