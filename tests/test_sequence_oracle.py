"""Pins of the sequence operators' 64-bit definitions (CPU): closed forms,
complex products, torch autograd, central differences, planted mistakes."""
import math

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as S

RNG = np.random.default_rng(7)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product(layout):
    x = RNG.standard_normal((5, 3, 12))
    pos = np.array([0, 1, 7, 1000, -3])
    y = S.rotate(x, pos, 8, layout, magnitude=1.5)
    a, b = (x[..., :4], x[..., 4:8]) if layout == "half" else (x[..., 0:8:2], x[..., 1:8:2])
    z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, None] * 10000.0 ** (-2.0 * np.arange(4) / 8))
    ya, yb = (y[..., :4], y[..., 4:8]) if layout == "half" else (y[..., 0:8:2], y[..., 1:8:2])
    assert np.allclose(ya, z.real, atol=1e-13) and np.allclose(yb, z.imag, atol=1e-13)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    # the transposed map: <R x, y> = <x, R^T y>; without magnitude it is the inverse
    u = RNG.standard_normal(x.shape)
    assert math.isclose((y * u).sum(), (x * S.rotate(u, pos, 8, layout, inverse=True, magnitude=1.5)).sum(), rel_tol=1e-12)
    back = S.rotate(S.rotate(x, pos, 8, layout), pos, 8, layout, inverse=True)
    assert np.allclose(back, x, atol=1e-13)


def test_frequencies():
    f = S.frequencies(64)
    assert f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64))
    assert np.allclose(S.frequencies(64, scaling="linear", factor=4.0), f / 4)
    # a larger base keeps the fastest pair and stretches the slowest by the factor
    b = S.frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1.0 and math.isclose(b[31], f[31] / 8, rel_tol=1e-12)
    for scaling in ("parts", "bands"):
        p = S.frequencies(64, scaling=scaling, factor=16.0, original_len=8192.0, turns_low=1.0, turns_high=32.0)
        turns = 8192 * f / (2 * math.pi)
        assert np.array_equal(p[turns >= 32], f[turns >= 32])
        assert np.allclose(p[turns <= 1], f[turns <= 1] / 16)
        mid = (turns > 1) & (turns < 32)
        assert mid.any() and ((p[mid] < f[mid]) & (p[mid] > f[mid] / 16)).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("weights", [True, False])
def test_gradient_against_autograd_and_differences(layout, weights):
    T, H, D, rot = 3, 2, 10, 6
    x, dy = RNG.standard_normal((T, H, D)), RNG.standard_normal((T, H, D))
    w = 1 + 0.3 * RNG.standard_normal(D) if weights else None
    pos = np.array([0, 5, 901])
    kw = dict(rot=rot, layout=layout, magnitude=1.2)
    dx, dw = S.norm_rotary_grad(x, dy, pos, w, 1e-3, **kw)
    tx = torch.tensor(x, requires_grad=True)
    tw = torch.tensor(np.ones(D) if w is None else w, requires_grad=True)
    n = tx * (tx.pow(2).mean(-1, keepdim=True) + 1e-3).rsqrt() * tw
    f = torch.tensor(S.frequencies(rot))
    ang = torch.tensor(pos)[:, None, None] * f
    a, b = (n[..., :3], n[..., 3:6]) if layout == "half" else (n[..., 0:6:2], n[..., 1:6:2])
    ya, yb = (a * ang.cos() - b * ang.sin()) * 1.2, (a * ang.sin() + b * ang.cos()) * 1.2
    y = torch.cat([ya, yb], -1) if layout == "half" else torch.stack([ya, yb], -1).flatten(-2)
    (torch.cat([y, n[..., 6:]], -1) * torch.tensor(dy)).sum().backward()
    assert np.allclose(dx, tx.grad.numpy(), atol=1e-12) and np.allclose(dw, tw.grad.numpy(), atol=1e-12)
    loss = lambda v: (S.norm_rotary(v, pos, w, 1e-3, **kw) * dy).sum()
    for i in ((0, 0, 0), (1, 1, 4), (2, 0, 9)):
        e = np.zeros_like(x)
        e[i] = 1e-5
        assert math.isclose((loss(x + e) - loss(x - e)) / 2e-5, dx[i], rel_tol=1e-6, abs_tol=1e-8)


def dense(q, keys, values, scale):
    s = scale * q @ keys.T
    p = np.exp(s - s.max())
    return p @ values / p.sum(), s.max() + math.log(p.sum())


def attention_inputs():
    page, hk, D = 4, 2, 6
    kc, vc = RNG.standard_normal((12, page, hk, D)), RNG.standard_normal((12, page, hk, D))
    perm = RNG.permutation(12)
    return dict(q=RNG.standard_normal((5, 4, D)), kc=kc, vc=vc, scale=0.4, offsets=[0, 2, 2, 5], lens=[5, 0, 3],
                table=perm[:6].reshape(3, 2), group_offsets=[0, 2, 3], prefix_lens=[7, 0], prefix_table=perm[6:10].reshape(2, 2))


def test_attention_against_dense_rows():
    a = attention_inputs()
    out, lse, bound = S.prefix_attention(**a)
    flat = lambda c, row, n, h: c[row].reshape(-1, 2, 6)[:n, h]
    for t, (b, seen, pre) in enumerate([(0, 4, 7), (0, 5, 7), (2, 1, 0), (2, 2, 0), (2, 3, 0)]):
        g = 0 if b < 2 else 1
        for h in range(4):
            keys = np.concatenate([flat(a["kc"], a["prefix_table"][g], pre, h // 2), flat(a["kc"], a["table"][b], seen, h // 2)])
            vals = np.concatenate([flat(a["vc"], a["prefix_table"][g], pre, h // 2), flat(a["vc"], a["table"][b], seen, h // 2)])
            o, z = dense(a["q"][t, h], keys, vals, 0.4)
            assert np.allclose(out[t, h], o, atol=1e-12) and math.isclose(lse[t, h], z, rel_tol=1e-12)
            assert (bound[t, h] >= np.abs(out[t, h]) - 1e-12).all()


def test_attention_empty_rows_and_bad_masks():
    a = attention_inputs()
    a["lens"] = [1, 0, 0]     # the first query of sequence 0 and all of sequence 2 see no own slot
    out, lse, _ = S.prefix_attention(**a)
    assert np.isfinite(lse[0]).all()          # it sees the prefix
    assert np.isneginf(lse[2:]).all() and (out[2:] == 0).all()
    assert S.slots([0, 2, 2, 5], [5, 0, 3]) == [(0, 3), (0, 4), (2, 0), (2, 1), (2, 2)]


def test_attention_catches_planted_mistakes():
    a = attention_inputs()
    out, lse, _ = S.prefix_attention(**a)
    for change in (dict(lens=[6, 0, 3]), dict(prefix_lens=[6, 0]), dict(scale=0.41), dict(group_offsets=[0, 3, 3]),
                   dict(table=a["table"][:, ::-1]), dict(kc=a["kc"][:, :, ::-1])):
        o2, l2, _ = S.prefix_attention(**{**a, **change})
        assert np.abs(o2 - out).max() > 1e-3 and np.abs(l2 - lse).max() > 1e-3, change
