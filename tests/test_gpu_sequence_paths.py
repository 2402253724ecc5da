"""GPU tests of the sequence operators' paths that follow from a call's size: groups of four heads and stores past
the L2 in large calls, tiles of 128 rows with the own slots taken along, results written without partial outputs,
parts of a prefix longer than a block's window of pages. Each test first makes sure, from sizes or from what the
workspace holds afterwards, that its call takes the path. Tolerances as in test_gpu_sequence.py; the definitions
are computed in 64 bits on the device here, since the calls are large."""
import math

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from oracle import sequence_oracle as S
from tests.test_gpu_sequence import DT, TINY, U, attention_case, half, i32, spec_of

pytestmark = pytest.mark.gpu


def draw(gen, shape, dt):
    return torch.randn(shape, generator=gen, device="cuda").to(DT[dt])


def near(got, want, err, dt, what):
    got = got.double()
    off = ~((got - want).abs() <= err + half(dt) * (1 + 1e-3) * want.abs() + TINY[dt])
    if off.any():
        i = tuple(int(x) for x in off.nonzero()[0])
        raise AssertionError(f"{what}: {int(off.sum())} of {off.numel()} off, first at {i}: {got[i]} for {want[i]}")


# ---- rotation and norm in groups of four heads -----------------------------------------------

def pairs(x, rot, layout):
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def unpair(a, b, rest, layout):
    turned = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def rotate64(x, pos, rot, layout, inverse=False, magnitude=1.0, **spec):
    f = torch.tensor(S.frequencies(rot, **spec), device="cuda")
    ang = pos.double()[:, None, None] * f
    c, s = magnitude * ang.cos(), magnitude * ang.sin() * (-1 if inverse else 1)
    a, b = pairs(x, rot, layout)
    return unpair(a * c - b * s, a * s + b * c, x[..., rot:], layout)


def pair_size(x, rot, layout, magnitude=1.0):
    a, b = pairs(x.abs(), rot, layout)
    return unpair(a + b, a + b, x[..., rot:].abs(), layout) * max(1.0, magnitude)


def norm64(x, w, eps=1e-6):
    return x * (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * (1.0 if w is None else w.double())


# dtype, layout, scaling, dim, rot, q heads, k heads, tokens, elements that the outputs start behind a line
BIG = [
    ("bf16", "half", "none", 128, 128, 6, 3, 14999, 0),         # whole lines: stores pass the L2 by
    ("bf16", "half", "none", 128, 128, 6, 3, 14999, 8),         # the same, 16 bytes behind a line
    ("bf16", "half", "parts", 128, 128, 5, 0, 27001, 0),
    ("f32", "half", "none", 64, 64, 6, 3, 14999, 0),
    ("f16", "half", "linear", 256, 256, 2, 3, 13999, 0),
    ("bf16", "interleaved", "none", 128, 128, 5, 1, 22003, 0),
    ("f16", "half", "parts", 96, 48, 5, 2, 25013, 0),
    ("f32", "interleaved", "bands", 64, 32, 7, 2, 15013, 0),
]
BIG_IDS = ["-".join(str(x) for x in c) for c in BIG]


def big_operands(case, seed):
    dt, layout, scaling, D, rot, hq, hk, T, behind = case
    V2 = 8 if dt == "f32" else 16
    assert T * (hq + hk) * (D // V2) >= 1 << 20 and D % V2 == 0 and rot % V2 == 0, "not the large calls' path"
    gen = torch.Generator(device="cuda").manual_seed(seed)
    fused = draw(gen, (T, hq + 2 * hk, D), dt)
    pos = torch.randint(0, 1 << 17, (T,), generator=gen, device="cuda")
    w = [1 + 0.2 * torch.randn(D, generator=gen, device="cuda") for _ in range(2)]

    def out(heads):
        flat = torch.full((T * heads * D + 64,), 7.0, dtype=DT[dt], device="cuda")
        assert flat.data_ptr() % 128 == 0
        return flat[behind:behind + T * heads * D].view(T, heads, D)

    return gen, fused[:, :hq], fused[:, hq:hq + hk], pos, w, out, spec_of(scaling, rot, layout)


@pytest.mark.parametrize("case", BIG, ids=BIG_IDS)
@pytest.mark.parametrize("normed", [True, False])
def test_large_rotation_and_norm(case, normed):
    dt, layout, _, D, rot, hq, hk, T, _ = case
    _, q, k, pos, w, out, spec = big_operands(case, 81)
    mag = spec.get("magnitude", 1.0)
    r = E.Rotary(**spec)
    qo, ko = out(hq), out(hk)
    args = (r.handle, pos, q, qo, k if hk else None, ko if hk else None)
    if normed:
        E.emb_qk_norm_rotary(*args, *w, 1e-6)
    else:
        E.emb_rotary_apply(*args)
    torch.cuda.synchronize()
    for name, x, y, wt in (("q", q, qo, w[0]), ("k", k, ko, w[1])):
        if x.shape[1] == 0:
            continue
        n = norm64(x.double(), wt) if normed else x.double()
        near(y, rotate64(n, pos, **spec), (24 if normed else 8) * U * pair_size(n, rot, layout, mag), dt, name)
        if not normed:
            assert torch.equal(y[..., rot:], x[..., rot:])
    # in place gives the same bits
    again = q.clone(), k.clone()
    args = (r.handle, pos, again[0], again[0], *((again[1], again[1]) if hk else (None, None)))
    if normed:
        E.emb_qk_norm_rotary(*args, *w, 1e-6)
    else:
        E.emb_rotary_apply(*args)
    assert torch.equal(again[0], qo) and (hk == 0 or torch.equal(again[1], ko))


@pytest.mark.parametrize("case", BIG, ids=BIG_IDS)
def test_large_gradient(case):
    dt, layout, _, D, rot, hq, hk, T, _ = case
    gen, q, k, pos, w, out, spec = big_operands(case, 82)
    mag = spec.get("magnitude", 1.0)
    dyq, dyk = draw(gen, (T, hq, D), dt), draw(gen, (T, hk, D), dt)
    r = E.Rotary(**spec)
    dq, dk = out(hq), out(hk)
    ws = torch.full((E.emb_qk_norm_rotary_workspace_bytes(T, hq, hk, D),), 255, dtype=torch.uint8, device="cuda")
    dwq, dwk = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
    E.emb_qk_norm_rotary_backward(r.handle, pos, q, dyq, dq, k if hk else None, dyk if hk else None,
                                  dk if hk else None, *w, 1e-6, ws, dwq, dwk)
    torch.cuda.synchronize()
    for name, x, dy, dx, wt, dw in (("q", q, dyq, dq, w[0], dwq), ("k", k, dyk, dk, w[1], dwk)):
        if x.shape[1] == 0:
            assert (dw == 0).all()
            continue
        x, dy, wt = x.double(), dy.double(), wt.double()
        u = rotate64(dy, pos, inverse=True, **spec)
        inv = (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
        n = x * inv
        g = u * wt
        size = pair_size(dy, rot, layout, mag)
        near(dx, inv * (g - n * (g * n).mean(-1, keepdim=True)),
             40 * U * inv * (size * wt.abs() + n.abs() * (size * wt.abs() * n.abs()).mean(-1, keepdim=True)), dt, "d" + name)
        near(dw, (u * n).sum((0, 1)), 100 * U * (size * n.abs()).sum((0, 1)), "f32", "dw" + name)


@pytest.mark.parametrize("dt,layout,scaling,D,rot,hk,page,normed", [
    ("bf16", "half", "none", 128, 128, 6, 16, True), ("bf16", "interleaved", "bands", 128, 64, 3, 64, True),
    ("f16", "half", "parts", 96, 48, 5, 32, False), ("f32", "half", "linear", 64, 64, 7, 7, True),
    ("bf16", None, None, 128, 0, 6, 16, False),
])
def test_large_append(dt, layout, scaling, D, rot, hk, page, normed):
    gen = torch.Generator(device="cuda").manual_seed(83)
    rng = np.random.default_rng(83)
    V2 = 8 if dt == "f32" else 16
    T = (1 << 20) // (2 * hk * (D // V2)) + 777
    assert T * 2 * hk * (D // V2) >= 1 << 20
    counts = [int(n) for n in np.diff(np.concatenate([[0], np.sort(rng.choice(T, 10)), [T]]))]
    lens = [n + int(h) for n, h in zip(counts, rng.integers(0, 200, len(counts)))]
    pages = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(pages)), -1, np.int32)
    pool = rng.permutation(sum(pages) + 3)
    at = np.concatenate([[0], np.cumsum(pages)])
    for b, n in enumerate(pages):
        table[b, :n] = pool[at[b]:at[b] + n]
    mk = lambda: draw(gen, (len(pool), hk, page, D), dt).transpose(1, 2)
    kc, vc = mk(), mk()
    k0, v0 = kc.clone(), vc.clone()
    x = draw(gen, (T, 2 * hk, D), dt)
    k, v = x[:, :hk], x[:, hk:]
    w = 1 + 0.2 * torch.randn(D, generator=gen, device="cuda") if normed else None
    off = np.concatenate([[0], np.cumsum(counts)])
    r = E.Rotary(**spec_of(scaling, rot, layout)) if layout else None
    cache = E.KVCache(kc, vc)
    E.emb_kv_append(cache.handle, r.handle if r else None, k, v, i32(off), i32(lens), torch.from_numpy(table).cuda(),
                    wk=w, eps=1e-6 if normed else None)
    cache.check_error()
    seq, slot = (torch.tensor(t).cuda() for t in zip(*S.slots(off, lens)))
    pg, sl = torch.from_numpy(table).cuda().long()[seq, slot // page], slot % page
    n = norm64(k.double(), w) if normed else k.double()
    if layout:
        spec = spec_of(scaling, rot, layout)
        near(kc[pg, sl], rotate64(n, slot, **spec), 24 * U * pair_size(n, rot, layout, spec.get("magnitude", 1.0)), dt, "keys")
    else:
        assert torch.equal(kc[pg, sl], k)
    k0[pg, sl], v0[pg, sl] = kc[pg, sl], v
    assert torch.equal(kc, k0) and torch.equal(vc, v0), "values are copied, no other slot changes"


# ---- attention ---------------------------------------------------------------------------------

def case_of(dt, D, hq, hk, page, counts, lens, sizes, prefix, **kw):
    """attention_case with an own table as wide as the own sequences need, not as the prefixes do."""
    q, kc, vc, off, lens, table, groups = attention_case(dt, D, hq, hk, page, counts, lens, sizes, prefix, **kw)
    return q, kc, vc, off, lens, table[:, :max(1, -(-max(lens) // page))].contiguous(), groups


class Call:
    """One call's sizes, and runs of it."""

    def __init__(self, q, kc, vc, off, lens, table, groups, scale):
        self.q, self.kc, self.vc, self.off, self.table, self.groups, self.scale = q, kc, vc, off, table, groups, scale
        self.lens = list(lens)
        self.cache = E.KVCache(kc, vc)
        T, hq, D = q.shape
        go, pl, pt = groups
        m = hq // kc.shape[2]
        self.wide = T * m > 64 * pl.numel() and kc.shape[1] % 8 == 0
        assert table.shape[1] * kc.shape[1] <= 256, "own slots would get blocks of their own"
        self.size = E.emb_prefix_attention_workspace_bytes(self.cache.handle, T, hq, pl.numel(), pt.shape[1], table.shape[1])
        self.parts = self.size // (T * hq * (D + 1) * 4) - 1      # of the prefix; one more is reserved for own blocks

    def run(self, lens=None, out=None):
        T, hq, D = self.q.shape
        ws = torch.full((self.size,), 255, dtype=torch.uint8, device="cuda")
        out = torch.full((T, hq, D), 7.0, dtype=self.q.dtype, device="cuda") if out is None else out
        lse = torch.full((T, hq), 7.0, device="cuda")
        E.emb_prefix_attention(self.cache.handle, self.q, out, self.scale, i32(self.off), i32(lens or self.lens), self.table,
                               *self.groups, ws, lse=lse)
        self.cache.check_error()
        # one part: nothing is written but the result
        assert bool((ws == 255).all()) == (self.parts == 1)
        return out, lse

    def check(self, out, lse, dt):
        want, wl, bound = attention64(self.q, self.kc, self.vc, self.scale, self.off, self.lens, self.table, self.groups)
        D, m = self.q.shape[2], self.q.shape[1] // self.kc.shape[2]
        kmax = self.kc.float().abs().nan_to_num(0, 0, 0).amax(dim=(0, 1)).double().repeat_interleave(m, 0)
        e = (D + 8) * U * abs(self.scale) * (self.q.double().abs() * kmax).sum(-1)
        near(out, want, (half(dt) + 2 * e[..., None] + 128 * U) * bound, dt, "out")
        assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
        live = ~torch.isneginf(wl)
        assert ((lse.double() - wl).abs() <= e + 256 * U + 4 * U * wl.abs())[live].all()


def attention64(q, kc, vc, scale, off, lens, table, groups):
    """The definition, group by group and head by head."""
    T, hq, D = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    m = hq // hk
    go, pl, pt = ([int(x) for x in groups[0]], [int(x) for x in groups[1]], groups[2].long())
    out, bound = torch.zeros((T, hq, D), dtype=torch.float64, device="cuda"), torch.zeros((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), float("-inf"), dtype=torch.float64, device="cuda")
    seq = np.repeat(np.arange(len(lens)), np.diff(off))
    seen = np.array([lens[b] - (off[b + 1] - off[b]) + t - off[b] + 1 for t, b in enumerate(seq)])
    W = max(1, max(lens))
    spot = torch.arange(W, device="cuda")
    own = table.long().clamp(min=0)[:, spot // page]
    for g in range(len(pl)):
        at = torch.arange(pl[g], device="cuda")
        pages = pt[g][at // page]
        t0, t1 = int(off[go[g]]), int(off[go[g + 1]])
        for a in range(t0, t1, 256):
            z = slice(a, min(a + 256, t1))
            where = own[torch.tensor(seq[z], device="cuda")]
            hide = spot[None] >= torch.tensor(seen[z], device="cuda")[:, None]
            for h in range(hk):
                kp, vp = kc[pages, at % page, h].double(), vc[pages, at % page, h].double()
                ko, vo = kc[where, spot % page, h].double(), vc[where, spot % page, h].double()
                for i in range(h * m, (h + 1) * m):
                    x = q[z, i].double()
                    s0 = scale * (x @ kp.t().contiguous())
                    s1 = (scale * (x[:, None] * ko).sum(-1)).masked_fill(hide, float("-inf"))
                    s = torch.cat([s0, s1], 1)
                    top = torch.logsumexp(s, 1)
                    p = torch.exp(s - torch.where(torch.isneginf(top), torch.zeros_like(top), top)[:, None])
                    p0, p1 = p[:, :pl[g]], p[:, pl[g]:]
                    out[z, i] = p0 @ vp + (p1[..., None] * vo).sum(1)
                    bound[z, i] = p0 @ vp.abs() + (p1[..., None] * vo.abs()).sum(1)
                    lse[z, i] = top
    return out, lse, bound


# name: (q heads per cache head, page, counts, lens, group sizes, prefixes, tiles of 128 rows, parts of the prefix)
TAKEN_ALONG = {
    "wide_direct": (32, 16, [1, 2] * 20, [9, 16] * 20, [25, 15], [170, 33], True, 1),
    "wide_parts": (4, 16, [1, 3] * 40, [5, 40] * 40, [50, 30], [1500, 700], True, None),
    "wide_many_groups": (32, 16, [2] * 80, [16, 5] * 40, [1] * 70 + [0, 10], [17] * 40 + [90] * 32, True, 1),
    "narrow_direct": (32, 7, [1, 2] * 20, [5, 7] * 20, [25, 15], [180, 33], False, 1),
    "narrow_parts": (2, 16, [1, 2] * 10, [9, 40] * 10, [20], [1500], False, None),
    "narrow_many_groups": (2, 16, [2] * 80, [16, 5] * 40, [1] * 70 + [0, 10], [17] * 40 + [90] * 32, False, None),
}


def along(kind, dt, D):
    m, page, counts, lens, sizes, prefix, wide, parts = TAKEN_ALONG[kind]
    c = Call(*case_of(dt, D, 2 * m, 2, page, counts, lens, sizes, prefix), 0.125)
    assert c.wide == wide and (c.parts == parts if parts else c.parts > 1), (c.wide, c.parts)
    return c, counts


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 96)])
@pytest.mark.parametrize("kind", list(TAKEN_ALONG))
def test_own_slots_taken_along(dt, D, kind):
    c, counts = along(kind, dt, D)
    base, base_l = c.run()
    c.check(base, base_l, dt)
    again, again_l = c.run()
    assert torch.equal(again, base) and torch.equal(again_l, base_l), "reruns are bit-identical"
    # into strided rows, whose other half stays
    out = torch.full((*base.shape[:2], 2 * D), 5.0, dtype=base.dtype, device="cuda")
    c.run(out=out[..., D:])
    assert torch.equal(out[..., D:], base) and (out[..., :D] == 5.0).all()
    # sequence 7's own slots hold infinities, NaN and huge keys: only its rows may notice
    page = c.kc.shape[1]
    own = [int(x) for x in c.table[7][:-(-c.lens[7] // page)]]
    t0, t1 = int(c.off[7]), int(c.off[8])
    rest = torch.ones(base.shape[0], dtype=torch.bool, device="cuda")
    rest[t0:t1] = False
    k1, v1 = c.kc.clone(), c.vc.clone()
    for poison in (float("nan"), float("inf"), torch.finfo(DT[dt]).max):
        c.kc[own], c.vc[own] = poison, poison
        got, got_l = c.run()
        assert torch.equal(got[rest], base[rest]) and torch.equal(got_l[rest], base_l[rest]), poison
        c.kc.copy_(k1), c.vc.copy_(v1)
    # an infinite value that only its last query sees
    assert counts[7] > 1
    c.vc[int(c.table[7][(c.lens[7] - 1) // page]), (c.lens[7] - 1) % page] = float("inf")
    got, got_l = c.run()
    rest[t0:t1 - 1] = True
    assert torch.equal(got[rest], base[rest]) and torch.equal(got_l, base_l)
    assert torch.isposinf(got[t1 - 1]).all()
    c.vc.copy_(v1)
    # its length is its own matter too
    other = list(c.lens)
    other[7] = counts[7]
    got, got_l = c.run(lens=other)
    rest[t0:t1] = False
    assert torch.equal(got[rest], base[rest]) and torch.equal(got_l[rest], base_l[rest])


def test_many_groups_write_their_results_directly():
    # tiles enough that a prefix is one part whatever its length; groups in no order
    rng = np.random.default_rng(91)
    counts = [2] * 1100
    lens = [int(n) for n in rng.integers(2, 41, len(counts))]
    cuts = np.sort(rng.choice(np.arange(1, 1100), 11, replace=False))
    sizes = [int(n) for n in np.diff(np.concatenate([[0], cuts, [1100]]))]
    c = Call(*case_of("bf16", 128, 32, 8, 16, counts, lens, sizes, [int(n) for n in rng.integers(0, 700, 12)]), 0.09)
    assert c.wide and c.parts == 1
    out, lse = c.run()
    c.check(out, lse, "bf16")


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 96), ("f16", 128), ("bf16", 64)])
def test_parts_longer_than_a_window_of_pages(dt, D):
    # a block looks up the pages of 1024 slots (heads of 96 and 128) or 2048 (64) at a time
    c = Call(*case_of(dt, D, 128, 32, 16, [1] * 256, [1 + i % 7 for i in range(256)], [256], [8999]), 1 / math.sqrt(D))
    assert c.wide and 8999 // c.parts > 2 * 2048, c.parts
    out, lse = c.run()
    c.check(out, lse, dt)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 96)])
@pytest.mark.parametrize("kind", ["wide", "narrow"])
def test_slots_behind_a_prefix_are_not_seen(dt, D, kind):
    # ends at many places of a tile, the slots behind them in the same page with infinities and NaN
    m = 32 if kind == "wide" else 2
    prefix = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 200, 255]
    G = len(prefix)
    c = Call(*case_of(dt, D, 2 * m, 2, 128, [3] * G, [3 + 5 * i for i in range(G)], [1] * G, prefix), 0.125)
    assert c.wide == (kind == "wide")
    base, base_l = c.run()
    c.check(base, base_l, dt)
    seen = torch.zeros(c.kc.shape[:2], dtype=torch.bool)
    for row, n in [(c.groups[2][g], prefix[g]) for g in range(G)] + [(c.table[b], c.lens[b]) for b in range(G)]:
        for s in range(n):
            seen[int(row[s // 128]), s % 128] = True
    assert 0.2 < seen.float().mean() < 0.9
    for poison in (float("nan"), float("inf"), torch.finfo(DT[dt]).min):
        c.kc[~seen.cuda()] = poison
        c.vc[~seen.cuda()] = poison
        got, got_l = c.run()
        assert torch.equal(got, base) and torch.equal(got_l, base_l), poison
