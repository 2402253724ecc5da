"""Plain CPU definitions of the sequence operators in 64 bits (numpy): rotary
positions, the per-head norm of queries and keys and its gradient, the append
to a paged cache, and the attention over a shared prefix. Loops over tokens
and heads, no code shared with the library. ``|.|`` companions give the
magnitudes that error bounds are scaled by."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, turns_low=0.0, turns_high=0.0,
                **_):
    """Radians per position of each pair."""
    out = []
    b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
    for i in range(rot // 2):
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling in ("parts", "bands"):
            turns = original_len * f / (2 * math.pi)
            if scaling == "parts":
                keep = math.log(turns / turns_low) / math.log(turns_high / turns_low)
            else:
                keep = (turns - turns_low) / (turns_high - turns_low)
            keep = min(1.0, max(0.0, keep))
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return np.array(out)


def rotate(x, positions, rot, layout, inverse=False, magnitude=1.0, **spec):
    """x [tokens, heads, dim] in 64 bits; the transposed map if inverse."""
    x = np.asarray(x, np.float64)
    f = frequencies(rot, **spec)
    y = x.copy()
    for t, pos in enumerate(np.asarray(positions, np.int64)):
        for i in range(rot // 2):
            ang = float(pos) * f[i]
            c, s = magnitude * math.cos(ang), magnitude * math.sin(ang)
            if inverse:
                s = -s
            a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return y


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r if w is None else x * r * np.asarray(w, np.float64)


def norm_rotary(x, positions, w, eps, **spec):
    return rotate(norm(x, w, eps), positions, **spec)


def norm_rotary_grad(x, dy, positions, w, eps, **spec):
    """(dx, dw) of norm_rotary."""
    x = np.asarray(x, np.float64)
    u = rotate(dy, positions, inverse=True, **spec)
    wv = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    g = u * wv
    return r * (g - n * (g * n).mean(-1, keepdims=True)), (u * n).sum((0, 1))


def slots(offsets, lens):
    """(sequence, slot) of every new token."""
    return [(b, int(lens[b]) - (int(offsets[b + 1]) - int(offsets[b])) + j)
            for b in range(len(lens)) for j in range(int(offsets[b + 1]) - int(offsets[b]))]


def prefix_attention(q, kc, vc, scale, offsets, lens, table, group_offsets=None, prefix_lens=None,
                     prefix_table=None):
    """q [tokens, q_heads, dim]; kc, vc [pages, page, heads, dim]. (out, lse, bound): bound is
    sum_j p_j |v_j|, which rounding errors of the products are relative to."""
    q, kc, vc = (np.asarray(a, np.float64) for a in (q, kc, vc))
    T, hq, D = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    out, bound = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse = np.full((T, hq), -np.inf)
    group = {}
    if prefix_lens is not None:
        for g in range(len(prefix_lens)):
            for b in range(int(group_offsets[g]), int(group_offsets[g + 1])):
                group[b] = g
    for b in range(len(lens)):
        n = int(offsets[b + 1]) - int(offsets[b])
        for j in range(n):
            t = int(offsets[b]) + j
            rows = []
            if b in group:
                g = group[b]
                rows += [(int(prefix_table[g][s // page]), s % page) for s in range(int(prefix_lens[g]))]
            rows += [(int(table[b][s // page]), s % page) for s in range(int(lens[b]) - n + j + 1)]
            if not rows:
                continue
            pg, sl = np.array(rows).T
            for h in range(hq):
                kk, vv = kc[pg, sl, h // (hq // hk)], vc[pg, sl, h // (hq // hk)]
                s = scale * (kk @ q[t, h])
                top = s.max()
                if top == -np.inf:
                    continue
                p = np.exp(s - top)
                lse[t, h] = top + math.log(p.sum())
                p /= p.sum()
                out[t, h] = p @ vv
                bound[t, h] = p @ np.abs(vv)
    return out, lse, bound
