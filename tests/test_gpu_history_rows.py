"""GPU tests of layer norm, its gradient and dropout against their 64-bit definitions (oracle/history_oracle.py).

Tolerances follow from the arithmetic, with u = 2^-24 (half an fp32 step) and h = eps / 2 of the result's type:
  - a row's sum is a chain of at most 16 terms in a lane and a tree of at most 6 + 16 more: 40 u of the mean of
    magnitudes, e_m = 40 u mean|x| absolute in the mean and in each difference, besides u |x - m| for its rounding;
  - the reciprocal deviation r is off by 50 u relative (sum of squares, quotient, root, quotient) and by what the
    differences' error moves it: d = 50 u + 2 r e_m;
  - y = ((x - m) r) w + b: |h w| (d + 4 u) + r |w| e_m + 2 u |b|, and the last rounding, h |y|;
  - with G = |g| + mean|g| + |h| mean|g h| the gradient is off by r G (d + 100 u) and by what h's error moves the
    product h mean(g h): r 2 mean|g| (d |h| + r e_m), and its last rounding;
  - dw: each term is off by |dy| (|h| (d + 4 u) + r e_m); the sum is a chain of rows in a group (at most `chain`), a
    tree of 3 + 4 and fp64: (chain + 10) u of the sum of magnitudes; db likewise;
  - dropout: a product and a sum, 3 u (|x| / (1 - p) + |residual|), and the last rounding.
"""
import gc
import threading

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from oracle import history_oracle as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half of the smallest step


@pytest.fixture(autouse=True)
def _free_gpu():
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def n64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, err, dt, what):
    got = n64(got)
    tol = err + torch.finfo(DT[dt]).eps / 2 * np.abs(want) * (1 + 1e-3) + TINY[dt]
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {tol[i]}")


def rows_of(gen, rows, dim, dt, memory, mean=0.5):
    x = torch.randn((rows, dim), generator=gen) * (0.1 + 2 * torch.rand((rows, 1), generator=gen))
    x = (x + mean * torch.randn((rows, 1), generator=gen)).to(DT[dt])
    if memory == "strided":     # a slice of wider rows, 16-byte aligned
        wide = torch.full((rows, dim + 24), float("nan"), dtype=DT[dt], device="cuda")
        out = wide[:, 8:8 + dim]
    elif memory == "odd":       # rows off 16-byte borders
        out = torch.full((rows, dim + 3), float("nan"), dtype=DT[dt], device="cuda")[:, 1:1 + dim]
    else:
        out = torch.empty((rows, dim), dtype=DT[dt], device="cuda")
    out.copy_(x)
    return out


# (x type, y type, rows, dim, memory)
NORM_CASES = [
    ("bf16", "bf16", 4, 64, "plain"), ("f32", "f32", 33, 128, "plain"), ("f32", "bf16", 70, 128, "plain"),
    ("f32", "f16", 9, 32, "plain"), ("f16", "f16", 257, 512, "strided"), ("bf16", "bf16", 19, 1024, "plain"),
    ("bf16", "bf16", 1, 8, "plain"), ("f32", "f32", 5, 4, "plain"), ("f32", "bf16", 3, 1, "plain"),
    ("bf16", "bf16", 300, 65, "plain"), ("f16", "f16", 7, 1000, "odd"), ("f32", "f32", 130, 7, "odd"),
    ("f32", "f16", 65, 96, "odd"), ("bf16", "bf16", 6, 1032, "plain"), ("f32", "f32", 5, 4096, "plain"),
    ("f16", "f16", 3, 4104, "strided"), ("bf16", "bf16", 2, 16384, "plain"), ("f32", "bf16", 2, 16383, "plain"),
    ("bf16", "bf16", 3, 2047, "odd"), ("f32", "f32", 20000, 16, "plain"), ("bf16", "bf16", 9001, 128, "strided"),
]


@pytest.mark.parametrize("xt,yt,rows,dim,memory", NORM_CASES)
@pytest.mark.parametrize("weights", [True, False])
def test_layer_norm_and_gradient(xt, yt, rows, dim, memory, weights):
    gen = torch.Generator().manual_seed(rows * 7919 + dim)
    x, dy = rows_of(gen, rows, dim, xt, memory), rows_of(gen, rows, dim, yt, memory)
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).cuda() if weights else None
    b = torch.randn(dim, generator=gen).cuda() if weights else None
    y, dx = rows_of(gen, rows, dim, yt, memory), rows_of(gen, rows, dim, xt, memory)
    E.emb_layer_norm(x, y, w, b, 1e-5)
    X, W, B, DY = n64(x), n64(w) if weights else np.ones(dim), n64(b) if weights else np.zeros(dim), n64(dy)
    want, m, r, h = H.layer_norm(X, W, B, 1e-5)
    em = 40 * U * np.abs(X).mean(1, keepdims=True) + U * np.abs(X - m)
    d = 50 * U + 2 * r * em.max(1, keepdims=True)
    close(y, want, np.abs(h * W) * (d + 4 * U) + r * np.abs(W) * em + 2 * U * np.abs(B), yt, "y")

    ws = torch.full((E.emb_layer_norm_workspace_bytes(rows, dim),), 0x7f, dtype=torch.uint8, device="cuda")
    dw, db = torch.full((dim,), 7.0, device="cuda"), torch.full((dim,), 7.0, device="cuda")
    E.emb_layer_norm_backward(x, dy, dx, w, 1e-5, ws, dw, db)
    wdx, wdw, wdb = H.layer_norm_backward(X, DY, W, 1e-5)
    g = np.abs(DY * W)
    big = g + g.mean(1, keepdims=True) + np.abs(h) * (g * np.abs(h)).mean(1, keepdims=True)
    err = r * big * (d + 100 * U) + r * 2 * g.mean(1, keepdims=True) * (d * np.abs(h) + r * em) + \
        r * np.abs(h) * (g * r * em).mean(1, keepdims=True)
    close(dx, wdx, err, xt, "dx")
    chain = 64
    close(dw, wdw, (np.abs(DY) * (np.abs(h) * (d + 4 * U) + r * em)).sum(0) + (chain + 10) * U * np.abs(DY * h).sum(0),
          "f32", "dw")
    close(db, wdb, (chain + 10) * U * np.abs(DY).sum(0), "f32", "db")
    # again: the same bits; without the weights' gradients and in place of dy too
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    E.emb_layer_norm_backward(x, dy, dx2, w, 1e-5, ws, dw2, db2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    dx3 = torch.empty_like(dx)
    E.emb_layer_norm_backward(x, dy, dx3, w, 1e-5, ws)
    assert torch.equal(dx, dx3)
    if xt == yt:
        E.emb_layer_norm_backward(x, dy, dy, w, 1e-5, ws, None, db2)
        assert torch.equal(dy, dx) and torch.equal(db, db2)
        E.emb_layer_norm(x, x, w, b, 1e-5)
        assert torch.equal(x, y)
    if memory != "plain":      # nothing beside the rows was written
        for t in (x, y, dx):
            rest = t._base.clone()
            rest[:, t.storage_offset():t.storage_offset() + dim] = float("nan")
            assert rest.isnan().all()


def test_layer_norm_without_rows():
    x = torch.empty((0, 64), device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    E.emb_layer_norm(x, x, None, None, 1e-5)
    E.emb_layer_norm_backward(x, x, x, None, 1e-5, torch.empty(16, dtype=torch.uint8, device="cuda"), dw, None)
    assert (dw == 0).all()


def test_layer_norm_of_constant_rows_and_of_specials():
    x = torch.full((4, 128), 3.0, device="cuda")
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    y = torch.empty_like(x)
    E.emb_layer_norm(x, y, None, torch.arange(128.0, device="cuda"), 1e-5)
    assert torch.equal(y[0], torch.arange(128.0, device="cuda")) and torch.equal(y[3], y[0])
    assert y[1].isnan().any() and y[2].isnan().all()


def test_layer_norm_broadcast_rows_and_one_row_weights():
    gen = torch.Generator().manual_seed(4)
    row = rows_of(gen, 1, 256, "bf16", "plain")
    x = row.expand(500, 256)
    y, one = torch.empty((500, 256), dtype=torch.bfloat16, device="cuda"), torch.empty_like(row)
    E.emb_layer_norm(x, y, None, None, 1e-5)
    E.emb_layer_norm(row, one, None, None, 1e-5)
    assert torch.equal(y, one.expand(500, 256))


# ---- dropout --------------------------------------------------------------------

DROP_CASES = [
    ("f32", 5, 64, "plain", 0.3, True), ("bf16", 33, 128, "plain", 0.1, True), ("f16", 9, 72, "strided", 0.5, False),
    ("bf16", 7, 65, "plain", 0.2, True), ("f32", 300, 3, "odd", 0.6, True), ("f16", 1, 1, "plain", 0.5, False),
    ("f32", 41, 130, "odd", 0.01, False), ("bf16", 12, 200, "strided", 0.0, True), ("f16", 12, 40, "plain", 1.0, True),
    ("f32", 3, 1001, "plain", 0.9, True),
]


@pytest.mark.parametrize("dt,rows,dim,memory,p,residual", DROP_CASES)
@pytest.mark.parametrize("step", [None, 0, 5 + (3 << 32) + (1 << 63)])
def test_dropout(dt, rows, dim, memory, p, residual, step):
    gen = torch.Generator().manual_seed(rows + dim)
    x, r, y = (rows_of(gen, rows, dim, dt, memory) for _ in range(3))
    seed = 0xDEADBEEF12345678
    at = None if step is None else torch.tensor([step - (1 << 64) if step >> 63 else step], device="cuda")
    E.emb_dropout(x, y, p, seed, step=at, residual=r if residual else None)
    want = H.dropout(n64(x), n64(r) if residual else None, p, seed, step or 0)
    mag = np.abs(n64(x)) / (1 if p == 1 else 1 - p) + (np.abs(n64(r)) if residual else 0)
    close(y, want, 3 * U * mag, dt, "y")
    kept = H.dropout_bits(rows, dim, seed, step or 0) >= np.uint64(int(p * 2 ** 32 + 0.5))
    if not residual:
        assert ((n64(y) != 0) == (kept & (n64(x) != 0))).all()
    y2 = x if p < 0.4 else r     # in place of an input
    E.emb_dropout(x, y2, p, seed, step=at, residual=r if residual else None)
    assert torch.equal(y, y2)
    if memory != "plain":
        rest = y._base.clone()
        rest[:, y.storage_offset():y.storage_offset() + dim] = float("nan")
        assert rest.isnan().all()


@pytest.mark.parametrize("dt,dim", [("f32", 64), ("bf16", 64), ("f16", 61)])
def test_dropout_ties_are_decided_by_the_lower_half(dt, dim):
    """A threshold at an element's own 32 bits keeps it, one above drops it."""
    bits = H.dropout_bits(40, dim, 77, 9)
    x = torch.ones((40, dim), dtype=DT[dt], device="cuda")
    y = torch.empty_like(x)
    step = torch.tensor([9], device="cuda")
    for r, c in ((0, 0), (3, 17), (39, dim - 1)):
        for over in (0, 1):
            E.emb_dropout(x, y, (int(bits[r, c]) + over) / 2 ** 32, 77, step=step)
            assert bool(y[r, c] != 0) == (over == 0)


def test_dropped_places_have_no_influence():
    bits = H.dropout_bits(16, 64, 5, 0)
    kept = torch.from_numpy(bits >= np.uint64(1 << 31)).cuda()
    x = torch.where(kept, 1.0, float("nan")).to(torch.bfloat16)
    x[~kept & (torch.arange(64, device="cuda") % 2 == 0)] = float("inf")
    y = torch.empty_like(x)
    E.emb_dropout(x, y, 0.5, 5, residual=torch.ones_like(x))
    assert torch.equal(y, torch.where(kept, 3.0, 1.0).to(torch.bfloat16))


def test_dropout_gradient_has_the_same_mask():
    gen = torch.Generator().manual_seed(1)
    x, dy = rows_of(gen, 50, 96, "f32", "plain"), rows_of(gen, 50, 96, "f32", "plain")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    E.emb_dropout(x, y, 0.4, 3)
    E.emb_dropout(dy, dx, 0.4, 3)
    # linear in x: the product with dy is the product of x with the gradient
    assert torch.equal(y != 0, dx != 0)
    assert abs((y.double() * dy.double()).sum() - (x.double() * dx.double()).sum()) < 1e-4


def test_graph_draws_another_mask_on_each_replay():
    x = torch.ones((64, 256), dtype=torch.bfloat16, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(256, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.empty(E.emb_layer_norm_workspace_bytes(64, 256), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)

    def run():
        E.emb_dropout(x, y, 0.5, 11, step=step)
        E.emb_layer_norm(y, z, w, None, 1e-5)
        E.emb_layer_norm_backward(y, z, dx, w, 1e-5, ws, dw)
        step.add_(1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    step.zero_()
    masks = []
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, z, dx, dw)]
        masks.append(got[0] != 0)
        assert int(step) == i + 1
        step.fill_(i)
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, z, dx, dw)):
            assert torch.equal(a, b)
    assert all(not torch.equal(a, b) for a, b in zip(masks, masks[1:]))


def test_other_streams_and_threads():
    gen = torch.Generator().manual_seed(2)
    x = rows_of(gen, 4000, 512, "bf16", "plain")
    ref, got = torch.empty_like(x), [torch.empty_like(x) for _ in range(4)]
    E.emb_layer_norm(x, ref, None, None, 1e-5)
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            if i % 2:
                E.emb_layer_norm(x, got[i], None, None, 1e-5, stream=s)
            else:
                with torch.cuda.stream(s):
                    E.emb_layer_norm(x, got[i], None, None, 1e-5)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all(torch.equal(g, ref) for g in got)


def test_many_rows_and_a_stride_beyond_32_bits():
    """Rows whose elements lie past 2^31: the offsets are 64-bit."""
    base = torch.empty(2 * (1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((3, 64), (1 << 31, 1))
    x.copy_(torch.randn((3, 64), device="cuda"))
    y, want = torch.empty((3, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 64), dtype=torch.bfloat16, device="cuda")
    E.emb_layer_norm(x, y, None, None, 1e-5)
    E.emb_layer_norm(x.contiguous(), want, None, None, 1e-5)
    assert torch.equal(y, want)
    E.emb_dropout(x, y, 0.3, 4)
    E.emb_dropout(x.contiguous(), want, 0.3, 4)
    assert torch.equal(y, want)
