"""Plain CPU definitions of the history layer's operators in 64 bits (numpy):
layer norm and its gradient, the dropout mask, buckets of distances, and the
attention of a ragged batch of histories with a bias by relative position, its
gradient and its form over a paged cache. Loops over rows, sequences and heads,
no code shared with the library."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def layer_norm(x, w, b, eps):
    """(y, m, r, h) of rows x; w and b may be None."""
    x = np.asarray(x, np.float64)
    m = x.mean(1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    h = (x - m) * r
    y = h * (1.0 if w is None else np.asarray(w, np.float64)) + (0.0 if b is None else np.asarray(b, np.float64))
    return y, m, r, h


def layer_norm_backward(x, dy, w, eps):
    """(dx, dw, db)."""
    dy = np.asarray(dy, np.float64)
    _, _, r, h = layer_norm(x, None, None, eps)
    g = dy * (1.0 if w is None else np.asarray(w, np.float64))
    dx = r * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


# ---- dropout -----------------------------------------------------------------

def philox(counter, key, rounds=10):
    """Philox4x32 in Python integers: four words for a counter of four and a key of two."""
    a, b, c, d = counter
    k0, k1 = key
    low = 2 ** 32 - 1
    for _ in range(rounds):
        x, y = 0xD2511F53 * a, 0xCD9E8D57 * c
        a, b, c, d = (y >> 32) ^ b ^ k0, y & low, (x >> 32) ^ d ^ k1, x & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return a, b, c, d


def dropout_bits(rows, dim, seed, step):
    """The 32 random bits of each element."""
    key = (seed % 2 ** 32, seed >> 32)
    out = np.zeros((rows, dim), np.uint64)
    for r in range(rows):
        for u in range(-(-dim // 8)):
            c2, c3 = step % 2 ** 32, (step >> 32) % 2 ** 31
            first, second = philox((u, r, c2, c3), key), philox((u, r, c2, c3 + 2 ** 31), key)
            for j in range(min(8, dim - 8 * u)):
                shift = 16 * (j % 2)
                hi, lo = first[j // 2] >> shift & 0xFFFF, second[j // 2] >> shift & 0xFFFF
                out[r, 8 * u + j] = hi << 16 | lo
    return out


def dropout(x, residual, p, seed, step):
    x = np.asarray(x, np.float64)
    t = int(p * 2 ** 32 + 0.5)
    kept = dropout_bits(*x.shape, seed, step) >= np.uint64(t)
    y = np.where(kept, x, 0.0) / (1.0 if t == 2 ** 32 else 1.0 - t / 2 ** 32)
    return y if residual is None else y + np.asarray(residual, np.float64)


# ---- attention ----------------------------------------------------------------

HIDDEN = -2.0 ** 13


def bucket(d, buckets, exact, far):
    """Bucket of a distance d >= 0, by exact comparisons."""
    if d < exact:
        return int(d)
    n = buckets - exact
    if n == 0:
        return buckets - 1
    k = 0
    while k + 1 < n and Fraction(int(d), exact) ** n >= Fraction(far, exact) ** (k + 1):
        k += 1
    return exact + k


def bias_row(delta, buckets, exact, far, causal):
    row = bucket(abs(delta), buckets, exact, far)
    return row + buckets if delta < 0 and not causal else row


def scores(q, k, scale, causal, bias, spec, first=0):
    """Scores [n, m] of queries at places first .. over keys at 0 .., and the bias' row of each pair; bias: [rows]."""
    n, m = len(q), len(k)
    s = np.asarray(q, np.float64) @ np.asarray(k, np.float64).T * scale
    rows = np.zeros((n, m), np.int64)
    delta = first + np.arange(n)[:, None] - np.arange(m)[None, :]
    if bias is not None:
        by = {int(d): bias_row(int(d), *spec, causal) for d in np.unique(delta)}
        rows = np.vectorize(by.get)(delta)
        b = np.asarray(bias, np.float64)
        s = s + np.where(b <= HIDDEN, -np.inf, b)[rows]
    if causal:
        s = np.where(delta < 0, -np.inf, s)
    return s, rows


def softmax(s):
    """(P, lse); rows that see nothing are zeros and -inf."""
    top = s.max(1, keepdims=True)
    e = np.exp(s - np.where(np.isneginf(top), 0.0, top))
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total[:, 0] > 0, np.log(total[:, 0]) + top[:, 0], -np.inf)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0), lse


def _product(p, x):
    """p @ x where a weight of zero takes nothing."""
    if np.isfinite(x).all():
        return p @ x
    out = np.zeros((p.shape[0], x.shape[1]))
    for i in range(p.shape[0]):
        for j in np.nonzero(p[i])[0]:
            out[i] = out[i] + p[i, j] * x[j]
    return out


def attention(q, k, v, offsets, scale, causal, bias=None, spec=None):
    """(out, lse, |P| |v|) of [tokens, heads, dim] arrays in 64 bits."""
    T, hq, D = q.shape
    m = hq // k.shape[1]
    out, lse, mag = np.zeros((T, hq, D)), np.full((T, hq), -np.inf), np.zeros((T, hq, D))
    for a, b in zip(offsets[:-1], offsets[1:]):
        if a == b:
            continue
        for h in range(hq):
            s, _ = scores(q[a:b, h], k[a:b, h // m], scale, causal, None if bias is None else bias[:, h], spec)
            p, lse[a:b, h] = softmax(s)
            out[a:b, h] = _product(p, v[a:b, h // m])
            mag[a:b, h] = _product(p, np.abs(v[a:b, h // m]))
    return out, lse, mag


def attention_backward(q, k, v, dout, offsets, scale, causal, bias=None, spec=None):
    """dict of dq, dk, dv, dbias, and of "|.|", the same sums over magnitudes (of dS: P (|dP| + sum P |dP|))."""
    T, hq, D = q.shape
    m = hq // k.shape[1]
    g = {n: np.zeros(s) for n, s in (("dq", q.shape), ("dk", k.shape), ("dv", v.shape))}
    g.update({"|" + n + "|": x.copy() for n, x in list(g.items())})
    if bias is not None:
        g["dbias"], g["|dbias|"] = np.zeros(bias.shape), np.zeros(bias.shape)
    for a, b in zip(offsets[:-1], offsets[1:]):
        if a == b:
            continue
        for h in range(hq):
            qs, ks, vs, do = q[a:b, h], k[a:b, h // m], v[a:b, h // m], dout[a:b, h]
            s, rows = scores(qs, ks, scale, causal, None if bias is None else bias[:, h], spec)
            p, _ = softmax(s)
            with np.errstate(invalid="ignore"):
                dp = np.where(p > 0, do @ vs.T, 0.0)
                adp = np.where(p > 0, np.abs(do) @ np.abs(vs).T, 0.0)
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            ads = p * (adp + (p * adp).sum(1, keepdims=True))
            for sign, x, key in ((ds, lambda t: t, "{}"), (ads, np.abs, "|{}|")):
                g[key.format("dq")][a:b, h] = _product(sign, x(ks)) * scale
                g[key.format("dk")][a:b, h // m] += _product(sign.T, x(qs)) * scale
                if bias is not None:
                    np.add.at(g[key.format("dbias")][:, h], rows, sign)
            g["dv"][a:b, h // m] += _product(p.T, do)
            g["|dv|"][a:b, h // m] += _product(p.T, np.abs(do))
    return g


def step(q, kc, vc, lens, table, scale, bias=None, spec=None):
    """(out, lse, |P| |v|) of one query for each sequence over its pages; caches [page, slot, head, dim]."""
    B, hq, D = q.shape
    page = kc.shape[1]
    m = hq // kc.shape[2]
    out, lse, mag = np.zeros((B, hq, D)), np.full((B, hq), -np.inf), np.zeros((B, hq, D))
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k = np.stack([kc[table[b, j // page], j % page] for j in range(n)])
        v = np.stack([vc[table[b, j // page], j % page] for j in range(n)])
        for h in range(hq):
            s, _ = scores(q[b, h:h + 1], k[:, h // m], scale, True, None if bias is None else bias[:, h], spec, n - 1)
            p, z = softmax(s)
            out[b, h], lse[b, h] = _product(p, v[:, h // m])[0], z[0]
            mag[b, h] = _product(p, np.abs(v[:, h // m]))[0]
    return out, lse, mag
