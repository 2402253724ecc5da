"""GPU tests of the layer over users' histories (dlrm_sparse_embedding_amd/history.py): layer norm, attention with a
bias by relative position, dropout, their gradients and the step over the paged cache together, as a training step and
serving use them. Each stage is held to its 64-bit definition on what the stage before it gave, so that its own rounding
counts alone; tolerances of layer norm and attention as in their own tests, with u = 2^-24 and h half a step of the
layer's type; a library product of n terms sums in fp32 and is rounded once: (n + 8) u of the sum of magnitudes, h of
the result; dropout and sum: 3 u of the magnitudes and h of the result."""
import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from dlrm_sparse_embedding_amd.history import HistoryEncoder
from oracle import history_oracle as H
from tests.test_gpu_history import Call, U, close, half, n64

pytestmark = pytest.mark.gpu

LENS = [70, 0, 1, 133, 40]
SPEC = (16, 8, 100)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def offsets_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


def encoder(dt="bf16", dim=64, heads=4, kv_heads=2, width=96, buckets=True, dropout=0.25):
    r = HistoryEncoder(300, width=width, heads=heads, kv_heads=kv_heads, dim=dim, buckets=SPEC[0] if buckets else 0,
                       exact=SPEC[1] if buckets else 0, far=SPEC[2] if buckets else 0, dropout=dropout, pages=64,
                       seed=(5 << 32) + 3, dtype={"bf16": torch.bfloat16, "f16": torch.float16}[dt])
    gen = torch.Generator().manual_seed(dim)
    r.tables.weights[0][0].copy_(torch.randn((300, width), generator=gen))
    r.norm_w.add_(0.2 * torch.randn(width, generator=gen).cuda())
    r.norm_b.add_(0.2 * torch.randn(width, generator=gen).cuda())
    if buckets:
        r.bias.copy_(torch.randn(r.bias.shape, generator=gen))
    r.count.fill_(7)
    return r, gen


def call_of(r, dt, fused, out, lse, lens, d_out=None):
    """The attention's operands as its own tests hold them."""
    c = Call.__new__(Call)
    c.dt, c.dim, c.hq, c.hk, c.causal, c.spec = dt, r.dim, r.heads, r.kv_heads, True, SPEC if r.bias is not None else None
    c.T, c.off, c.scale = sum(lens), [0, *np.cumsum(lens).tolist()], float(np.float32(r.dim ** -0.5))
    c.h, c.bias, c.out, c.lse, c.dout = r.attention, r.bias, out, lse, d_out
    c.q, c.k, c.v = r.parts(fused)
    c.offsets = offsets_of(lens)
    return c


def product(x, w):
    """A library product of 16-bit factors: the value and what its sum may be off by."""
    return x @ w, (x.shape[1] + 8) * U * (np.abs(x) @ np.abs(w))


@pytest.mark.parametrize("dt,dim,heads,kv_heads,width,buckets", [
    ("bf16", 64, 4, 2, 96, True), ("f16", 128, 2, 2, 64, True), ("bf16", 96, 3, 1, 200, False)])
def test_a_training_step(dt, dim, heads, kv_heads, width, buckets):
    r, gen = encoder(dt, dim, heads, kv_heads, width, buckets)
    h = half(dt)
    ids = torch.randint(0, 40, (sum(LENS),), generator=gen).cuda()      # some items many times
    offsets = offsets_of(LENS)
    rows = r.rows(ids)
    assert torch.equal(rows, r.tables.weights[0][0][ids])
    y, saved = r.forward(rows, offsets, train=True)
    _, _, normed, fused, out, lse = saved

    # forward
    X, W, B = n64(rows), n64(r.norm_w), n64(r.norm_b)
    want, m, rs, hx = H.layer_norm(X, W, B, 1e-5)
    em = 40 * U * np.abs(X).mean(1, keepdims=True) + U * np.abs(X - m)
    d = 50 * U + 2 * rs * em.max(1, keepdims=True)
    close(normed, want, np.abs(hx * W) * (d + 4 * U) + rs * np.abs(W) * em + 2 * U * np.abs(B), dt, "normed")
    want, err = product(n64(normed), n64(r.proj))
    close(fused.flatten(1), want, err, dt, "fused")
    dy = (torch.randn(y.shape, generator=gen)).to(y.dtype).cuda()
    d_back = torch.empty_like(dy)
    E.emb_dropout(dy, d_back, 0.25, r.seed, step=r.count)
    d_out = (d_back @ r.back.t()).view_as(out)
    c = call_of(r, dt, fused, out, lse, LENS, d_out)
    c.check_forward()
    want, err = product(n64(out).reshape(len(ids), -1), n64(r.back))
    err += h * np.abs(want)
    kept = H.dropout(np.ones(y.shape), None, 0.25, r.seed, 7)
    res = n64(rows.to(y.dtype))
    close(y, want * kept + res, (err + 3 * U * np.abs(want)) * kept + 3 * U * np.abs(res), dt, "y")

    # gradients
    want = n64(dy) * kept
    close(d_back, want, 3 * U * np.abs(want), dt, "d_back")
    want, err = product(n64(d_back), n64(r.back).T)
    close(d_out.flatten(1), want, err, dt, "d_out")
    grads = r.backward(saved, dy)
    g = torch.empty_like(fused)
    c.dq, c.dk, c.dv = r.parts(g)
    c.dbias = None if r.bias is None else torch.empty_like(r.bias)
    c.ws = torch.empty(E.emb_history_attention_workspace_bytes(r.attention.handle, c.T, len(LENS)), dtype=torch.uint8,
                       device="cuda")
    c.backward()
    c.check_backward()
    assert (grads["bias"] is None) if r.bias is None else torch.equal(grads["bias"], c.dbias)
    for name, a, b in (("proj", normed, g.flatten(1)), ("back", out.flatten(1), d_back)):
        want, err = product(n64(a).T, n64(b))
        close(grads[name], want, err, dt, name)
    d_normed = g.flatten(1) @ r.proj.t()
    want, err = product(n64(g).reshape(len(ids), -1), n64(r.proj).T)
    close(d_normed, want, err, dt, "d_normed")
    DY = n64(d_normed)
    dx, dw, db = H.layer_norm_backward(X, DY, W, 1e-5)
    gw = np.abs(DY * W)
    big = gw + gw.mean(1, keepdims=True) + np.abs(hx) * (gw * np.abs(hx)).mean(1, keepdims=True)
    err = rs * big * (d + 100 * U) + rs * 2 * gw.mean(1, keepdims=True) * (d * np.abs(hx) + rs * em) + \
        rs * np.abs(hx) * (gw * rs * em).mean(1, keepdims=True)
    close(grads["rows"], dx + n64(dy), err + U * np.abs(dx), "f32", "rows")
    close(grads["norm_w"], dw, (np.abs(DY) * (np.abs(hx) * (d + 4 * U) + rs * em)).sum(0) +
          74 * U * np.abs(DY * hx).sum(0), "f32", "norm_w")
    close(grads["norm_b"], db, 74 * U * np.abs(DY).sum(0), "f32", "norm_b")

    # the step: the same bits, taken from every weight
    names = {"proj": r.master, "back": r.back_master, "norm_w": r.norm_w, "norm_b": r.norm_b, "bias": r.bias}
    before = {n: w.clone() for n, w in names.items() if w is not None}
    table = r.tables.weights[0][0].clone()
    seen = []
    y2 = r.train_step(ids, offsets, lambda e: seen.append(e.clone()) or dy, lr=0.05)
    assert torch.equal(y2, y) and torch.equal(seen[0], y) and r.count.item() == 8
    for n, w in before.items():
        assert torch.equal(names[n], w - 0.05 * grads[n].float())
    assert torch.equal(r.proj, r.master.to(y.dtype)) and torch.equal(r.back, r.back_master.to(y.dtype))
    moved = (r.tables.weights[0][0] != table).any(1).nonzero().flatten()
    assert torch.equal(moved, torch.unique(ids))
    y3, _ = r.forward(r.rows(ids), offsets, train=True)
    assert not torch.equal(y3, y)
    r.attention.check_error()
    r.tables.check_device_error()
    r.close()


@pytest.mark.parametrize("dt,dim", [("bf16", 64), ("f16", 128)])
def test_serving_gives_the_last_rows_of_the_whole(dt, dim):
    """Histories appended but for their last three items, which follow one by one: each new row is that of the layer
    over the whole history."""
    r, gen = encoder(dt, dim)
    h = half(dt)
    lens = [40, 3, 133, 17]
    ids = [torch.randint(0, 300, (n,), generator=gen).cuda() for n in lens]
    table = r.new_pages(lens)
    held = [n - 3 for n in lens]
    first = r.append(torch.cat([x[:n] for x, n in zip(ids, held)]), offsets_of(held), i32(held), table)
    at = 0
    rows = r.rows(torch.cat(ids))
    whole, (_, _, _, fused, out, lse) = r.forward(rows, offsets_of(lens))
    c = call_of(r, dt, fused, out, lse, lens)
    c.check_forward()
    # both forms' outputs are within tol_out of the definition, then come two products and two last roundings
    o = n64(out).reshape(len(rows), -1)
    back = np.abs(n64(r.back))
    _, err = product(o, n64(r.back))
    tol = 2 * ((c.tol_out + h * np.abs(n64(out))).reshape(o.shape) @ back * (1 + 1e-3) + err + 2 * h * np.abs(o @ n64(r.back)))
    tol += 2 * 1.01 * h * np.abs(n64(whole)) + 2.0 ** -24
    start = np.cumsum([0, *lens])
    for u, n in enumerate(held):
        got = n64(first[at:at + n])
        assert (np.abs(got - n64(whole)[start[u]:start[u] + n]) <= tol[start[u]:start[u] + n]).all()
        at += n
    for more in range(3):
        now = [n + more + 1 for n in held]
        y = r.step(torch.stack([x[n - 1] for x, n in zip(ids, now)]), i32(now), table)
        at = [start[u] + n - 1 for u, n in enumerate(now)]
        assert (np.abs(n64(y) - n64(whole)[at]) <= tol[at]).all()
    r.cache.check_error()
    r.return_pages(table)
    r.close()


def test_captured_and_replayed():
    """Forward and gradient in a graph that counts its steps: each replay draws its own masks and equals the eager
    call of that step, with other work in between."""
    r, gen = encoder()
    ids = torch.randint(0, 300, (sum(LENS),), generator=gen).cuda()
    offsets, rows = offsets_of(LENS), r.rows(ids)
    dy = torch.randn((len(ids), 96), generator=gen).bfloat16().cuda()

    def work():
        y, saved = r.forward(rows, offsets, train=True)
        return y, r.backward(saved, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = work()
        r.count.add_(1)
    last = None
    for step in (7, 8, 9):
        assert r.count.item() == step
        graph.replay()
        torch.cuda.synchronize()
        assert r.count.item() == step + 1
        got = [y.clone()] + [g.clone() for g in grads.values()]
        r.count.fill_(step)
        eager = work()
        for a, b in zip(got, [eager[0], *eager[1].values()]):
            assert torch.equal(a, b)
        r.count.add_(1)
        assert last is None or not torch.equal(last, got[0])
        last = got[0]
        rows.mul_(0.5)
    r.close()


def test_two_layers_on_two_streams():
    """Training on one stream and serving on another at once: the bits of one after the other."""
    (a, gen), (b, _) = encoder(), encoder("bf16", 128)
    ids = torch.randint(0, 300, (sum(LENS),), generator=gen).cuda()
    offsets = offsets_of(LENS)
    dy = torch.randn((len(ids), 96), generator=gen).bfloat16().cuda()
    rows = a.rows(ids)
    lens = i32([max(n, 1) for n in LENS])
    new = ids[:len(LENS)]
    table = b.new_pages([n + 1 for n in LENS])
    b.append(ids, offsets, i32(LENS), table)

    def train():
        y, saved = a.forward(rows, offsets, train=True)
        return [y, *a.backward(saved, dy).values()]
    want_a, want_b = train(), b.step(new, lens, table)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got_a, got_b = [], []
    for _ in range(5):
        with torch.cuda.stream(one):
            got_a.append(train())
        with torch.cuda.stream(two):
            got_b.append(b.step(new, lens, table))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for got in got_a for x, w in zip(got, want_a))
    assert all(torch.equal(x, want_b) for x in got_b)
    a.close()
    b.close()
