"""Pins of the history layer's definitions (oracle/history_oracle.py) to torch's own functions, published numbers,
differences and closed forms (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import history_oracle as H


def test_layer_norm_is_torchs():
    rng = np.random.default_rng(0)
    x, w, b, dy = rng.normal(size=(7, 33)) + 3, rng.normal(size=33), rng.normal(size=33), rng.normal(size=(7, 33))
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], 1e-5)
    assert np.allclose(H.layer_norm(x, w, b, 1e-5)[0], y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(dy))
    for got, want in zip(H.layer_norm_backward(x, dy, w, 1e-5), t):
        assert np.allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("counter,key,want", [
    # known answers published with the generator
    ((0, 0, 0, 0), (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ((2 ** 32 - 1,) * 4, (2 ** 32 - 1,) * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0), "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_philox_known_answers(counter, key, want):
    assert " ".join(f"{w:08x}" for w in H.philox(counter, key)) == want


def test_dropout_keeps_the_stated_share():
    bits = H.dropout_bits(60, 200, 12345, 6)
    n = bits.size
    for p in (0.1, 0.5, 0.9):
        kept = (bits >= np.uint64(int(p * 2 ** 32))).mean()
        assert abs(kept - (1 - p)) < 5 * math.sqrt(p * (1 - p) / n)
    x = np.ones((3, 9))
    assert (H.dropout(x, None, 0.0, 1, 2) == 1).all() and (H.dropout(x, x, 1.0, 1, 2) == 1).all()


def test_buckets():
    # twice the distance every 8 buckets: borders that are whole numbers belong to the upper bucket
    assert [H.bucket(d, 32, 16, 64) for d in (0, 15, 16, 31, 32, 33, 63, 64, 10 ** 6)] == [0, 15, 16, 23, 24, 24, 31, 31, 31]
    assert [H.bucket(d, 4, 4, 0) for d in (0, 3, 4, 99)] == [0, 3, 3, 3]
    for buckets, exact, far in ((32, 16, 128), (64, 32, 1024), (7, 1, 100), (10, 3, 5)):
        last = 0
        for d in range(2 * far):
            b = H.bucket(d, buckets, exact, far)
            assert last <= b < buckets
            last = b
            if d >= exact:
                x = math.log(d / exact) / math.log(far / exact) * (buckets - exact)
                if abs(x - round(x)) > 1e-9:
                    assert b == min(buckets - 1, exact + math.floor(x))
    assert H.bias_row(-5, 32, 16, 128, False) == 37 and H.bias_row(5, 32, 16, 128, False) == 5


@pytest.mark.parametrize("causal", [True, False])
def test_attention_and_gradient_are_torchs(causal):
    gen = torch.Generator().manual_seed(3)
    T, hq, hk, D, spec = 23, 4, 2, 8, (8, 4, 12)
    off = [0, 0, 9, 10, 23]
    q, k, v, do = (torch.randn((T, h, D), generator=gen, dtype=torch.float64) for h in (hq, hk, hk, hq))
    bias = torch.randn((8 if causal else 16, hq), generator=gen, dtype=torch.float64)
    leaves = [t.requires_grad_() for t in (q, k, v, bias)]
    outs = []
    for a, b in zip(off[:-1], off[1:]):
        n = b - a
        rows = torch.tensor([[H.bias_row(i - j, *spec, causal) for j in range(n)] for i in range(n)], dtype=torch.int64)
        add = bias[rows.reshape(n, n)].permute(2, 0, 1)
        if causal:
            add = add.masked_fill(torch.ones(n, n).triu(1).bool(), float("-inf"))
        outs.append(torch.nn.functional.scaled_dot_product_attention(
            q[a:b].transpose(0, 1), k[a:b].transpose(0, 1).repeat_interleave(2, 0),
            v[a:b].transpose(0, 1).repeat_interleave(2, 0), add, scale=0.3).transpose(0, 1))
    out = torch.cat(outs)
    arrays = [t.detach().numpy() for t in (q, k, v)]
    got, lse, _ = H.attention(*arrays, off, 0.3, causal, bias.detach().numpy(), spec)
    assert np.allclose(got, out.detach().numpy(), atol=1e-12)
    assert np.isfinite(lse).all()
    out.backward(do)
    g = H.attention_backward(*arrays, do.numpy(), off, 0.3, causal, bias.detach().numpy(), spec)
    for name, t in zip(("dq", "dk", "dv", "dbias"), leaves):
        assert np.allclose(g[name], t.grad.numpy(), atol=1e-12), name
        assert (g[f"|{name}|"] >= np.abs(g[name]) - 1e-12).all()


def test_gradient_against_differences():
    rng = np.random.default_rng(5)
    q, k, v, do = (rng.normal(size=(6, 1, 4)) for _ in range(4))
    bias, off, spec = rng.normal(size=(3, 1)), [0, 6], (3, 2, 4)
    g = H.attention_backward(q, k, v, do, off, 0.5, True, bias, spec)

    def loss(**kw):
        a = dict(q=q, k=k, v=v, bias=bias, **{})
        a.update(kw)
        return (H.attention(a["q"], a["k"], a["v"], off, 0.5, True, a["bias"], spec)[0] * do).sum()
    for name, x in (("q", q), ("k", k), ("v", v), ("bias", bias)):
        for i in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[i] = 1e-6
            assert abs((loss(**{name: x + e}) - loss(**{name: x - e})) / 2e-6 - g["d" + name][i]) < 1e-7


def test_hidden_distances_and_empty_rows():
    rng = np.random.default_rng(6)
    q, k, v = (rng.normal(size=(5, 1, 4)) for _ in range(3))
    bias = np.array([[-np.inf], [0.0], [-3.4e38]])
    out, lse, _ = H.attention(q, k, v, [0, 5], 0.5, True, bias, (3, 3, 0))
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()          # sees only itself, at a hidden distance
    assert np.allclose(out[1:, 0], v[:-1, 0])                          # sees its neighbour alone
    g = H.attention_backward(q, k, v, rng.normal(size=(5, 1, 4)), [0, 5], 0.5, True, bias, (3, 3, 0))
    assert (g["dq"] == 0).all() and (g["dbias"] == 0).all()


def test_step_is_the_last_row():
    rng = np.random.default_rng(7)
    n, page = 21, 4
    q, k, v = (rng.normal(size=(n, h, 4)) for h in (2, 1, 1))
    bias, spec = rng.normal(size=(5, 2)), (5, 2, 9)
    table = rng.permutation(6)[None, :]
    kc, vc = np.zeros((6, page, 1, 4)), np.zeros((6, page, 1, 4))
    for j in range(n):
        kc[table[0, j // page], j % page], vc[table[0, j // page], j % page] = k[j], v[j]
    out, lse, _ = H.step(q[-1:], kc, vc, [n], table, 0.4, bias, spec)
    want, z, _ = H.attention(q, k, v, [0, n], 0.4, True, bias, spec)
    assert np.allclose(out[0], want[-1]) and np.allclose(lse[0], z[-1])


@pytest.mark.parametrize("planted", ["bias", "mask", "delta"])
def test_planted_mistakes_show(planted, monkeypatch):
    rng = np.random.default_rng(8)
    q, k, v, do = (rng.normal(size=(12, 1, 4)) for _ in range(4))
    bias, spec = rng.normal(size=(6, 1)), (6, 2, 10)
    good = H.attention(q, k, v, [0, 5, 12], 0.5, True, bias, spec)[0]
    if planted == "bias":
        old = H.bucket
        monkeypatch.setattr(H, "bucket", lambda d, *a: old(d + (d == 2), *a))
    if planted == "mask":
        assert not np.allclose(H.attention(q, k, v, [0, 5, 12], 0.5, False, np.concatenate([bias, bias]), spec)[0], good)
        return
    if planted == "delta":
        # without the row's sum the gradient of the bias does not sum to zero
        g = H.attention_backward(q, k, v, do, [0, 5, 12], 0.5, True, bias, spec)
        assert abs(g["dbias"].sum()) < 1e-12 < abs((g["|dbias|"]).sum())
        return
    assert not np.allclose(H.attention(q, k, v, [0, 5, 12], 0.5, True, bias, spec)[0], good)
