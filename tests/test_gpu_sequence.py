"""GPU tests of the sequence operators against their 64-bit definitions
(oracle/sequence_oracle.py).

Tolerances follow from the arithmetic, with u = 2^-24 (half an fp32 step) and
h = eps / 2 of the result's type (half a step):
  - a rotated element is two products and a sum of fp32 values, with sine and
    cosine within 4 u (series 5e-9, phase 2^-32 of a turn, conversions):
    8 u (|a| + |b|) magnitude, and h |y| for the last rounding;
  - the norm's factor is a sum of squares, a root and a quotient: 16 u more;
  - a gradient's element is a difference of two such terms: 40 u of the sum of
    their magnitudes; a weight's gradient is a sum of at most 64 terms in a
    lane's chain and a tree: 100 u of the sum of magnitudes;
  - an attention score is a sum of D products: e = (D + 8) u max_j scale |q|.|k_j|
    absolute, which moves probabilities by that much relative; probabilities
    are rounded to the cache's type (h) for the product with V:
    (h + 2 e + 128 u) sum_j p_j |v_j| and h |out|; lse: e + 256 u + 4 u |lse|.
"""
import gc
import math

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from oracle import sequence_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half of the smallest step

SPECS = {
    "none": dict(scaling="none", base=10000.0),
    "linear": dict(scaling="linear", base=10000.0, factor=4.0),
    "base": dict(scaling="base", base=10000.0, factor=8.0),
    "parts": dict(scaling="parts", base=10000.0, factor=16.0, original_len=8192.0, turns_low=1.0, turns_high=32.0,
                  magnitude=1.25),
    "bands": dict(scaling="bands", base=500000.0, factor=8.0, original_len=8192.0, turns_low=1.0, turns_high=4.0),
}


@pytest.fixture(autouse=True)
def _free_gpu():
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def half(dt):
    return torch.finfo(DT[dt]).eps / 2


def n64(t):
    return t.detach().double().cpu().numpy()


def randn(gen, shape, dt):
    return torch.randn(shape, generator=gen).to(DT[dt]).cuda()


def close(got, want, err, dt, what):
    got = n64(got)
    tol = err + half(dt) * np.abs(want) * (1 + 1e-3) + TINY[dt]
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(i)}: {got[tuple(i)]} "
                             f"for {want[tuple(i)]}, tolerance {tol[tuple(i)]}")


def pair_mag(x, rot, layout, magnitude=1.0):
    """|a| + |b| of each element's pair."""
    m = np.abs(n64(x)) if isinstance(x, torch.Tensor) else np.abs(x)
    out = m.copy()
    if layout == "half":
        s = m[..., :rot // 2] + m[..., rot // 2:rot]
        out[..., :rot // 2] = s
        out[..., rot // 2:rot] = s
    else:
        s = m[..., 0:rot:2] + m[..., 1:rot:2]
        out[..., 0:rot:2] = s
        out[..., 1:rot:2] = s
    return out * max(1.0, abs(magnitude))


# (dtype, layout, scaling, dim, rot, q heads, k heads, tokens, memory)
ROT_CASES = [
    ("bf16", "half", "none", 64, 64, 16, 4, 4, "fused"),
    ("bf16", "half", "none", 128, 128, 8, 2, 33, "fused"),
    ("f32", "interleaved", "linear", 64, 64, 4, 4, 70, "fused"),
    ("f16", "half", "parts", 96, 48, 6, 2, 41, "fused"),
    ("f16", "interleaved", "bands", 96, 96, 3, 1, 19, "plain"),
    ("bf16", "interleaved", "base", 128, 64, 5, 5, 7, "heads_first"),
    ("f32", "half", "none", 128, 32, 2, 1, 1, "plain"),
    ("f32", "half", "parts", 48, 16, 7, 3, 100, "plain"),
    ("bf16", "half", "none", 256, 256, 3, 1, 65, "plain"),
    ("bf16", "half", "none", 512, 64, 2, 2, 9, "plain"),
    ("f16", "half", "linear", 80, 80, 4, 2, 12, "plain"),
    ("bf16", "interleaved", "none", 16, 16, 3, 0, 300, "plain"),
    ("bf16", "half", "none", 72, 20, 3, 1, 11, "plain"),        # nothing divides 16 bytes
    ("f32", "interleaved", "bands", 7, 2, 2, 1, 5, "plain"),
    ("f16", "half", "none", 33, 30, 1, 1, 130, "odd"),
    ("bf16", "half", "none", 128, 128, 4, 2, 21, "odd"),        # a whole head, not on 16 bytes
    ("f32", "half", "base", 1000, 250, 2, 1, 3, "plain"),
    ("bf16", "half", "none", 1024, 256, 1, 1, 2, "plain"),
    ("f32", "half", "none", 64, 64, 0, 3, 17, "plain"),
]
IDS = ["-".join(str(x) for x in c) for c in ROT_CASES]


def views(gen, dt, T, hq, hk, D, memory):
    """q and k of one memory layout."""
    if memory == "fused":          # one projection's output: q, k and what follows
        x = randn(gen, (T, hq + 2 * hk, D), dt)
        return x[:, :hq], x[:, hq:hq + hk]
    if memory == "heads_first":    # [heads][tokens][dim]
        return randn(gen, (hq, T, D), dt).transpose(0, 1), randn(gen, (hk, T, D), dt).transpose(0, 1)
    if memory == "odd":            # rows one element apart from any alignment
        x = randn(gen, (T, hq + hk, D + 1), dt)
        return x[:, :hq, 1:], x[:, hq:, 1:]
    return randn(gen, (T, hq, D), dt), randn(gen, (T, hk, D), dt)


def positions(gen, T, kind):
    if kind == "i32":
        return torch.randint(0, 32768, (T,), generator=gen, dtype=torch.int32).cuda()
    p = torch.randint(-200000, 1 << 20, (T,), generator=gen, dtype=torch.int64)
    p[0] = 0
    return p.cuda()


def spec_of(scaling, rot, layout):
    return dict(rot=rot, layout=layout, **SPECS[scaling])


@pytest.mark.parametrize("case", ROT_CASES, ids=IDS)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(case, inverse):
    dt, layout, scaling, D, rot, hq, hk, T, memory = case
    gen = torch.Generator().manual_seed(11)
    q, k = views(gen, dt, T, hq, hk, D, memory)
    pos = positions(gen, T, "i64" if inverse else "i32")
    spec = spec_of(scaling, rot, layout)
    r = E.Rotary(**spec)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    E.emb_rotary_apply(r.handle, pos, q, qo, k if hk else None, ko if hk else None, inverse=inverse)
    torch.cuda.synchronize()
    mag = spec.get("magnitude", 1.0)
    # beyond 2^20 positions the 64-bit oracle's own angle is off by more; not drawn here
    for name, x, y in (("q", q, qo), ("k", k, ko)):
        if x.shape[1] == 0:
            continue
        want = S.rotate(n64(x), pos.cpu().numpy(), inverse=inverse, **spec)
        close(y, want, 8 * U * pair_mag(x, rot, layout, mag), dt, name)
        assert torch.equal(y[..., rot:], x[..., rot:]), "elements behind the rotation are copied"


@pytest.mark.parametrize("case", ROT_CASES, ids=IDS)
@pytest.mark.parametrize("weights", [True, False])
def test_norm_rotary(case, weights):
    dt, layout, scaling, D, rot, hq, hk, T, memory = case
    gen = torch.Generator().manual_seed(12)
    q, k = views(gen, dt, T, hq, hk, D, memory)
    pos = positions(gen, T, "i64")
    spec = spec_of(scaling, rot, layout)
    wq = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if weights else None
    wk = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if weights else None
    r = E.Rotary(**spec)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    E.emb_qk_norm_rotary(r.handle, pos, q, qo, k if hk else None, ko if hk else None, wq, wk, 1e-6)
    torch.cuda.synchronize()
    for name, x, y, w in (("q", q, qo, wq), ("k", k, ko, wk)):
        if x.shape[1] == 0:
            continue
        n = S.norm(n64(x), None if w is None else n64(w), 1e-6)
        want = S.rotate(n, pos.cpu().numpy(), **spec)
        close(y, want, 24 * U * pair_mag(n, rot, layout, spec.get("magnitude", 1.0)), dt, name)


@pytest.mark.parametrize("case", ROT_CASES, ids=IDS)
@pytest.mark.parametrize("weights", [True, False])
def test_norm_rotary_backward(case, weights):
    dt, layout, scaling, D, rot, hq, hk, T, memory = case
    gen = torch.Generator().manual_seed(13)
    q, k = views(gen, dt, T, hq, hk, D, memory)
    dyq, dyk = views(gen, dt, T, hq, hk, D, "plain" if memory == "odd" else memory)
    pos = positions(gen, T, "i64")
    spec = spec_of(scaling, rot, layout)
    mag = spec.get("magnitude", 1.0)
    wq = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if weights else None
    wk = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if weights else None
    r = E.Rotary(**spec)
    dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ws = torch.full((max(E.emb_qk_norm_rotary_workspace_bytes(T, hq, hk, D), 256),), 255, dtype=torch.uint8,
                    device="cuda")
    dwq, dwk = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")

    def run():
        E.emb_qk_norm_rotary_backward(r.handle, pos, q, dyq, dq, k if hk else None, dyk if hk else None,
                                      dk if hk else None, wq, wk, 1e-6, ws, dwq if weights else None,
                                      dwk if weights else None)
        torch.cuda.synchronize()

    run()
    p = pos.cpu().numpy()
    for name, x, dy, dx, w, dw in (("q", q, dyq, dq, wq, dwq), ("k", k, dyk, dk, wk, dwk)):
        x64, dy64 = n64(x), n64(dy)
        if x.shape[1] == 0:
            if weights:
                assert torch.equal(dw, torch.zeros_like(dw))
            continue
        w64 = None if w is None else n64(w)
        want, want_w = S.norm_rotary_grad(x64, dy64, p, w64, 1e-6, **spec)
        inv = 1.0 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-6)
        g = pair_mag(dy64, rot, layout, mag) * (1.0 if w64 is None else np.abs(w64))
        n = np.abs(x64 * inv)
        close(dx, want, 40 * U * inv * (g + n * (g * n).mean(-1, keepdims=True)), dt, "d" + name)
        if weights:
            bound = (pair_mag(dy64, rot, layout, mag) * n).sum((0, 1))
            close(dw, want_w, 100 * U * bound, "f32", "dw" + name)
    again = [t.clone() for t in (dq, dk, dwq, dwk)]
    run()
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert torch.equal(a, b), "reruns are bit-identical"


def test_rotary_many_tokens_and_in_place():
    # more heads than one wave of the chip takes, in place, against the same call out of place
    gen = torch.Generator().manual_seed(3)
    T, hq, hk, D = 5003, 8, 2, 128
    x = torch.randn((T, hq + 2 * hk, D), generator=gen).bfloat16().cuda()
    pos = torch.randint(0, 1 << 17, (T,), generator=gen).cuda()
    r = E.Rotary(128)
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    E.emb_qk_norm_rotary(r.handle, pos, q, qo, k, ko, w, w, 1e-6)
    some = [0, 1, 2500, 4096, 5002]
    n = S.norm(n64(q[some]), n64(w), 1e-6)
    want = S.rotate(n, pos[some].cpu().numpy(), rot=128, layout="half")
    close(qo[some], want, 24 * U * pair_mag(n, 128, "half"), "bf16", "q")
    kept = x[:, hq + hk:].clone()
    E.emb_qk_norm_rotary(r.handle, pos, q, q, k, k, w, w, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, hq + hk:], kept)


def test_norm_backward_many_tokens():
    gen = torch.Generator().manual_seed(4)
    T, hq, hk, D = 6001, 6, 2, 64
    q, k = randn(gen, (T, hq, D), "bf16"), randn(gen, (T, hk, D), "bf16")
    dyq, dyk = randn(gen, (T, hq, D), "bf16"), randn(gen, (T, hk, D), "bf16")
    pos = torch.arange(T).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    r = E.Rotary(64)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dwq, dwk = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(E.emb_qk_norm_rotary_workspace_bytes(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    E.emb_qk_norm_rotary_backward(r.handle, pos, q, dyq, dq, k, dyk, dk, w, w, 1e-6, ws, dwq, dwk)
    torch.cuda.synchronize()
    for x, dy, dx, dw in ((q, dyq, dq, dwq), (k, dyk, dk, dwk)):
        # rotation as a complex product, all in 64 bits on the device
        f = torch.tensor(S.frequencies(64), device="cuda")
        ang = pos.double()[:, None] * f
        z = torch.polar(torch.ones_like(ang), -ang)[:, None]
        u = torch.complex(dy[..., :32].double(), dy[..., 32:].double()) * z
        u = torch.cat([u.real, u.imag], -1)
        inv = (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
        n = x.double() * inv
        g = u * w.double()
        want = inv * (g - n * (g * n).mean(-1, keepdim=True))
        err = 40 * U * inv * (2 * g.abs() + 1 + n.abs() * (g * n).abs().mean(-1, keepdim=True) * 2)
        close(dx, n64(want), n64(err) + 40 * U * n64(inv) * n64(dy.abs().amax(-1, keepdim=True)), "bf16", "dx")
        close(dw, n64((u * n).sum((0, 1))), 100 * U * n64((u.abs() + dy.abs().double()).mul(n.abs()).sum((0, 1))),
              "f32", "dw")


def test_no_tokens_and_no_weights_gradient():
    r = E.Rotary(64)
    q = torch.empty((0, 4, 64), device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    E.emb_rotary_apply(r.handle, pos, q, q)
    dw = torch.full((64,), 3.0, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    E.emb_qk_norm_rotary_backward(r.handle, pos, q, q, q, q, q, q, None, None, 1e-6, ws, dw, dw.clone())
    torch.cuda.synchronize()
    assert torch.equal(dw, torch.zeros_like(dw))


# ---- the paged cache -----------------------------------------------------------------

def paged(gen, dt, pages, page, hk, D, order="heads_first"):
    if order == "heads_first":     # [page][head][slot][dim]
        mk = lambda: randn(gen, (pages, hk, page, D), dt).transpose(1, 2)
    elif order == "slots_first":
        mk = lambda: randn(gen, (pages, page, hk, D), dt)
    else:                          # a slice of wider rows
        pad = 8 if order == "padded" else 1
        mk = lambda: randn(gen, (pages, page, hk, D + pad), dt)[..., :D]
    return mk(), mk()


def page_table(rng, pages, page, lens, extra=1):
    """Shuffled pages, each used once; -1 past a sequence's last."""
    need = [-(-int(n) // page) for n in lens]
    perm = rng.permutation(pages)[:sum(need)]
    width = max(need + [0]) + extra
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).cuda()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


APPEND_CASES = [
    # dtype, layout, scaling, dim, rot, heads, page, norm, counts of new tokens, held before, order
    ("bf16", "half", "none", 128, 128, 8, 16, False, None, [0, 15, 16, 17, 100], "heads_first"),
    ("bf16", "interleaved", "bands", 128, 64, 8, 64, True, [70, 0, 1, 33, 0], [5, 64, 63, 0, 9], "heads_first"),
    ("f16", "half", "parts", 96, 48, 2, 32, True, [3, 40], [30, 0], "slots_first"),
    ("f32", "half", "linear", 64, 64, 1, 1, False, [2, 5, 1], [0, 3, 9], "heads_first"),
    ("f32", "interleaved", "none", 64, 32, 3, 7, True, [20, 9], [3, 14], "padded"),
    ("bf16", "half", "base", 72, 40, 3, 5, True, [11, 2], [1, 4], "odd"),
    ("bf16", None, None, 64, 0, 2, 16, False, [9, 20], [8, 0], "slots_first"),
    ("f16", None, None, 64, 0, 2, 16, True, [9, 20], [8, 0], "heads_first"),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=[f"{c[0]}-{c[1]}-{c[3]}-{c[6]}-{c[10]}-{c[7]}" for c in APPEND_CASES])
@pytest.mark.parametrize("given", [False, True])
def test_append(case, given):
    dt, layout, scaling, D, rot, hk, page, normed, new, held, order = case
    if given and layout is None:
        pytest.skip("positions go with a rotation")
    gen = torch.Generator().manual_seed(21)
    rng = np.random.default_rng(21)
    counts = new or [1] * len(held)
    lens = [h + c for h, c in zip(held, counts)]
    T = sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    pages = sum(-(-n // page) for n in lens) + 3
    kc, vc = paged(gen, dt, pages, page, hk, D, order)
    k0, v0 = kc.clone(), vc.clone()
    table = page_table(rng, pages, page, lens)
    x = randn(gen, (T, 2 * hk, D), dt)
    k, v = x[:, :hk], x[:, hk:]
    wk = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if normed else None
    spec = spec_of(scaling, rot, layout) if layout else None
    r = E.Rotary(**spec) if layout else None
    cache = E.KVCache(kc, vc)
    where = S.slots(off, lens)
    pos = torch.tensor([s + 1000 for _, s in where]).cuda() if given else None
    E.emb_kv_append(cache.handle, r.handle if r else None, k, v, None if new is None else i32(off), i32(lens), table,
                    wk=wk, eps=1e-6 if normed else None, positions=pos)
    cache.check_error()
    n = S.norm(n64(k), n64(wk), 1e-6) if normed else n64(k)
    p = [s + (1000 if given else 0) for _, s in where]
    want = S.rotate(n, p, **spec) if layout else n
    err = 24 * U * (pair_mag(n, rot, layout, spec.get("magnitude", 1.0)) if layout else np.abs(n))
    th = table.cpu().numpy()
    pg = torch.tensor([th[b, s // page] for b, s in where], dtype=torch.int64).cuda()
    sl = torch.tensor([s % page for _, s in where]).cuda()
    close(kc[pg, sl], want, err, dt, "keys")
    assert torch.equal(vc[pg, sl], v), "values are copied"
    k0[pg, sl], v0[pg, sl] = kc[pg, sl], v
    assert torch.equal(kc, k0) and torch.equal(vc, v0), "no other slot changes"


def test_append_skips_bad_slots_and_reports_them():
    gen = torch.Generator().manual_seed(22)
    kc, vc = paged(gen, "bf16", 4, 16, 2, 64)
    k0, v0 = kc.clone(), vc.clone()
    cache = E.KVCache(kc, vc)
    k, v = randn(gen, (5, 2, 64), "bf16"), randn(gen, (5, 2, 64), "bf16")
    # pages: outside the pool, negative, beyond the width, a slot below 0, and a good one
    table = torch.tensor([[4, 0], [-1, 0], [0, 1], [0, 1], [2, 3]], dtype=torch.int32).cuda()
    lens = i32([3, 3, 33, 0, 20])
    E.emb_kv_append(cache.handle, None, k, v, None, lens, table)
    with pytest.raises(E.EmbError) as ei:
        cache.check_error()
    assert ei.value.code == E.EMB_E_BOUNDS
    cache.check_error()   # reported once
    assert torch.equal(kc[3, 3], k[4]) and torch.equal(vc[3, 3], v[4])
    k0[3, 3], v0[3, 3] = k[4], v[4]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


# ---- attention --------------------------------------------------------------------------

def attention_tol(q, kc, vc, scale, lse, bound, dt, D):
    kmax = n64(kc.float().abs().nan_to_num(0, 0, 0).amax(dim=(0, 1)))            # [heads, D]: an upper bound of |k|
    m = q.shape[1] // kc.shape[2]
    e = (D + 8) * U * abs(scale) * (np.abs(n64(q)) * np.repeat(kmax, m, 0)).sum(-1)
    return (half(dt) + 2 * e[..., None] + 128 * U) * bound, e + 256 * U + 4 * U * np.abs(lse)


def run_attention(cache, q, scale, off, lens, table, groups=None, out=None, stream=None):
    T, hq, D = q.shape
    go, pl, pt = groups if groups else (None, None, None)
    n = E.emb_prefix_attention_workspace_bytes(cache.handle, T, hq, 0 if pl is None else pl.numel(),
                                               0 if pt is None else pt.shape[1], table.shape[1])
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")       # NaNs: nothing unwritten is used
    out = torch.full((T, hq, D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((T, hq), 7.0, device="cuda")
    E.emb_prefix_attention(cache.handle, q, out, scale, off, lens, table, go, pl, pt, ws, lse=lse, stream=stream)
    return out, lse


def check_attention(out, lse, q, kc, vc, scale, off, lens, table, groups, dt):
    D = q.shape[2]
    k64, v64 = n64(kc), n64(vc)
    want, wl, bound = S.prefix_attention(n64(q), k64, v64, scale, off, lens, table.cpu().numpy(),
                                         *([t.cpu().numpy() for t in groups] if groups else (None, None, None)))
    tol, tl = attention_tol(q, kc, vc, scale, np.where(np.isinf(wl), 0, wl), bound, dt, D)
    close(out, want, tol, dt, "out")
    got = n64(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(wl))
    live = ~np.isneginf(wl)
    assert (np.abs(got[live] - wl[live]) <= tl[live]).all(), np.abs(got[live] - wl[live]).max()


def attention_case(dt, D, hq, hk, page, counts, lens, group_sizes, prefix, seed=31, order="heads_first", big=1.0):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    T = sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    pages = sum(-(-n // page) for n in list(lens) + list(prefix)) + 3
    kc, vc = paged(gen, dt, pages, page, hk, D, order)
    both = page_table(rng, pages, page, list(prefix) + list(lens))
    G = len(prefix)
    q = (randn(gen, (T, hq, D), "f32") * big).to(DT[dt])
    groups = None
    if G:
        go = np.concatenate([[0], np.cumsum(group_sizes)])
        groups = (i32(go), i32(prefix), both[:G].contiguous())
    return q, kc, vc, off, lens, both[G:].contiguous(), groups


ATT_CASES = [
    # dtype, dim, hq, hk, page, counts, lens, group sizes, prefix lengths
    ("bf16", 128, 8, 2, 16, [1] * 8, [5, 1, 24, 16, 17, 32, 33, 7], [8], [200]),
    ("f16", 64, 4, 4, 32, [1] * 5, [1, 33, 2, 64, 65], [5], [511]),
    ("bf16", 128, 4, 1, 16, [2] * 6, [2, 40, 33, 17, 3, 32], [2, 0, 3, 1], [64, 100, 1, 31]),
    ("bf16", 96, 6, 2, 7, [3, 0, 1, 5], [9, 4, 1, 50], [1, 3], [0, 70]),
    ("f16", 128, 3, 1, 1, [1, 1], [1, 3], [2], [5]),
    ("bf16", 64, 40, 1, 64, [2, 1], [70, 3], [2], [130]),            # more query heads than a tile has rows
    ("bf16", 64, 64, 1, 16, [3], [40], [], []),                       # no prefix at all
    ("f16", 96, 10, 10, 16, [40, 7], [300, 7], [1, 1], [0, 33]),      # many own tokens: causal tiles
    ("bf16", 128, 8, 8, 16, [1] * 3, [0, 0, 0], [1, 2], [40, 0]),     # rows that see nothing
    ("bf16", 128, 2, 2, 16, [70], [70], [1], [300]),                  # a prompt behind a prefix
    ("f16", 64, 2, 2, 128, [1, 33], [600, 40], [2], [1000]),          # parts of prefix and own sequence
    ("bf16", 128, 4, 2, 16, [4], [2], [1], [33]),                     # more new tokens than the sequence holds
]


@pytest.mark.parametrize("case", ATT_CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}x{c[3]}-{c[4]}-{i}" for i, c in enumerate(ATT_CASES)])
@pytest.mark.parametrize("order", ["heads_first", "slots_first", "padded"])
def test_prefix_attention(case, order):
    dt, D, hq, hk, page, counts, lens, gs, prefix = case
    q, kc, vc, off, lens, table, groups = attention_case(*case, order=order)
    cache = E.KVCache(kc, vc)
    scale = 1.0 / math.sqrt(D)
    one = all(c == 1 for c in counts)
    out, lse = run_attention(cache, q, scale, None if one else i32(off), i32(lens), table, groups)
    cache.check_error()
    check_attention(out, lse, q, kc, vc, scale, off, lens, table, groups, dt)
    if one:   # the same with the offsets written out
        o2, l2 = run_attention(cache, q, scale, i32(off), i32(lens), table, groups)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_attention_ignores_what_a_query_does_not_see(dt):
    # infinities, NaN and the type's lowest value in every unseen slot: behind the ends, and
    # behind each query's own place among its sequence's new tokens
    case = (dt, 64, 4, 2, 16, [2, 1, 5], [18, 3, 40], [2, 1], [37, 70])
    q, kc, vc, off, lens, table, groups = attention_case(*case)
    cache = E.KVCache(kc, vc)
    base, base_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
    k1, v1 = kc.clone(), vc.clone()
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    both = [(groups[2][g], int(groups[1][g])) for g in range(2)] + [(table[b], lens[b]) for b in range(3)]
    for row, n in both:
        for s in range(n):
            seen[int(row[s // 16]), s % 16] = True
    for poison in (float("nan"), float("inf"), torch.finfo(DT[dt]).min):
        kc[~seen.cuda()] = poison
        vc[~seen.cuda()] = poison
        got, got_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
        assert torch.equal(got, base) and torch.equal(got_l, base_l)
    kc.copy_(k1), vc.copy_(v1)
    # the last slot of sequence 2 is seen by its last query only (token 7)
    pg, sl = int(table[2][39 // 16]), 39 % 16
    for poison in (float("nan"), float("inf")):
        kc[pg, sl] = poison
        vc[pg, sl] = poison
        got, got_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
        assert torch.equal(got[:7], base[:7]) and torch.equal(got_l[:7], base_l[:7])
        assert not torch.isfinite(got[7]).any()
        kc.copy_(k1), vc.copy_(v1)


def test_attention_with_large_scores():
    # scores of several hundred: the running maximum moves, nothing overflows
    case = ("bf16", 128, 4, 2, 16, [1, 2], [50, 9], [2], [700])
    q, kc, vc, off, lens, table, groups = attention_case(*case, big=40.0)
    cache = E.KVCache(kc, vc)
    out, lse = run_attention(cache, q, 0.3, i32(off), i32(lens), table, groups)
    check_attention(out, lse, q, kc, vc, 0.3, off, lens, table, groups, "bf16")


def exact_one_group(q, kc, vc, scale, lens, table, prefix, prefix_row):
    """64-bit attention of one-token sequences over one prefix, by head."""
    T, hq, D = q.shape
    hk, page = kc.shape[2], kc.shape[1]
    m = hq // hk
    out = torch.empty((T, hq, D), dtype=torch.float64, device="cuda")
    bound, lse = torch.empty_like(out), torch.empty((T, hq), dtype=torch.float64, device="cuda")
    at = torch.arange(prefix, device="cuda")
    pg = prefix_row.long()[at // page]
    W = max(lens)
    w = torch.arange(W, device="cuda")
    own = table.long().clamp(min=0)[:, w // page]
    hide = w[None] >= torch.tensor(lens, device="cuda")[:, None]
    for h in range(hk):
        kp, vp = kc[pg, at % page, h].double(), vc[pg, at % page, h].double()
        ko, vo = kc[own, w % page, h].double(), vc[own, w % page, h].double()     # [T, W, D]
        for i in range(h * m, (h + 1) * m):
            x = q[:, i].double()
            s0 = scale * (x @ kp.t().contiguous())
            s1 = (scale * (x[:, None] * ko).sum(-1)).masked_fill(hide, float("-inf"))
            z = torch.logsumexp(torch.cat([s0, s1], 1), 1)
            p0, p1 = torch.exp(s0 - z[:, None]), torch.exp(s1 - z[:, None])
            out[:, i] = p0 @ vp + (p1[..., None] * vo).sum(1)
            bound[:, i] = p0 @ vp.abs() + (p1[..., None] * vo.abs()).sum(1)
            lse[:, i] = z
    return n64(out), n64(lse), n64(bound)


@pytest.mark.parametrize("dt,D,hq,hk,page,seqs,prefix", [
    ("bf16", 128, 8, 2, 16, 8, 4096), ("f16", 64, 4, 4, 32, 301, 5003), ("bf16", 128, 8, 2, 64, 130, 9001),
    ("bf16", 96, 4, 2, 16, 64, 2999), ("f16", 128, 2, 1, 16, 1, 20011), ("bf16", 64, 16, 2, 48, 700, 777),
    ("f16", 128, 16, 2, 32, 40, 1500), ("f16", 96, 8, 1, 16, 333, 1025), ("bf16", 128, 4, 4, 16, 128, 64),
])
def test_attention_long_prefix(dt, D, hq, hk, page, seqs, prefix):
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(1, 40, seqs)]
    q, kc, vc, off, lens, table, groups = attention_case(dt, D, hq, hk, page, [1] * seqs, lens, [seqs], [prefix])
    cache = E.KVCache(kc, vc)
    scale = 1 / math.sqrt(D)
    out, lse = run_attention(cache, q, scale, None, i32(lens), table, groups)
    cache.check_error()
    want, wl, bound = exact_one_group(q, kc, vc, scale, lens, table, prefix, groups[2][0])
    tol, tl = attention_tol(q, kc, vc, scale, wl, bound, dt, D)
    close(out, want, tol, dt, "out")
    assert (np.abs(n64(lse) - wl) <= tl).all(), np.abs(n64(lse) - wl).max()
    o2, l2 = run_attention(cache, q, scale, None, i32(lens), table, groups)
    assert torch.equal(out, o2) and torch.equal(lse, l2), "reruns are bit-identical"


def test_attention_strided_operands_and_no_lse():
    case = ("bf16", 64, 4, 2, 16, [1] * 4, [3, 4, 5, 6], [4], [50])
    q, kc, vc, off, lens, table, groups = attention_case(*case)
    cache = E.KVCache(kc, vc)
    base, _ = run_attention(cache, q, 0.125, None, i32(lens), table, groups)
    wide = torch.empty((4, 8, 64), dtype=q.dtype, device="cuda")
    wide[:, :4] = q
    out = torch.full((4, 4, 128), 5.0, dtype=q.dtype, device="cuda")
    ws = torch.empty(E.emb_prefix_attention_workspace_bytes(cache.handle, 4, 4, 1, groups[2].shape[1], table.shape[1]),
                     dtype=torch.uint8, device="cuda")
    E.emb_prefix_attention(cache.handle, wide[:, :4], out[..., 64:], 0.125, None, i32(lens), table, *groups, ws)
    torch.cuda.synchronize()
    assert torch.equal(out[..., 64:], base)
    assert (out[..., :64] == 5.0).all()


def test_attention_reports_bad_pages_lengths_and_offsets():
    case = ("bf16", 64, 4, 2, 16, [1] * 4, [3, 4, 5, 6], [4], [50])
    q, kc, vc, off, lens, table, groups = attention_case(*case)
    cache = E.KVCache(kc, vc)
    base, _ = run_attention(cache, q, 0.125, None, i32(lens), table, groups)
    cache.check_error()

    def expect(code, lens_=lens, table_=table, groups_=groups, good=()):
        out, _ = run_attention(cache, q, 0.125, None, i32(lens_), table_, groups_)
        with pytest.raises(E.EmbError) as ei:
            cache.check_error()
        assert ei.value.code == code
        for t in good:
            assert torch.equal(out[t], base[t])

    t2 = table.clone()
    t2[1, 0] = kc.shape[0]
    expect(E.EMB_E_BOUNDS, table_=t2, good=(0, 2, 3))
    t2[1, 0] = -5
    expect(E.EMB_E_BOUNDS, table_=t2, good=(0, 2, 3))
    expect(E.EMB_E_BOUNDS, lens_=[3, 1 << 20, 5, 6], table_=table.clamp(min=0), good=(0, 2, 3))
    expect(E.EMB_E_BOUNDS, lens_=[3, -7, 5, 6], good=(0, 2, 3))
    p2 = groups[2].clone()
    p2[0, 1] = 1 << 30
    expect(E.EMB_E_BOUNDS, groups_=(groups[0], groups[1], p2))
    expect(E.EMB_E_BOUNDS, groups_=(groups[0], i32([1 << 29]), groups[2].clamp(min=0)))
    expect(E.EMB_E_INVAL, groups_=(i32([0, 3]), groups[1], groups[2]), good=(0, 1, 2))
    expect(E.EMB_E_INVAL, groups_=(i32([-4, 4000]), groups[1], groups[2]))


def test_append_then_attend_on_another_stream():
    gen = torch.Generator().manual_seed(41)
    rng = np.random.default_rng(41)
    hk, hq, D, page, B = 2, 8, 128, 16, 6
    lens = [int(x) for x in rng.integers(1, 40, B)]
    pages = sum(-(-n // page) for n in lens) + 20
    kc, vc = paged(gen, "bf16", pages, page, hk, D)
    table = page_table(rng, pages, page, lens)
    cache, r = E.KVCache(kc, vc), E.Rotary(D)
    x = randn(gen, (B, hq + 2 * hk, D), "bf16")
    w = torch.ones(D, device="cuda")
    pos = torch.tensor([n - 1 for n in lens]).cuda()

    def step(st):
        q = torch.empty((B, hq, D), dtype=torch.bfloat16, device="cuda")
        E.emb_qk_norm_rotary(r.handle, pos, x[:, :hq], q, None, None, w, None, 1e-6, stream=st)
        E.emb_kv_append(cache.handle, r.handle, x[:, hq:hq + hk], x[:, hq + hk:], None, lens_d, table, wk=w, eps=1e-6,
                        stream=st)
        return run_attention(cache, q, 0.1, None, lens_d, table, stream=st)

    lens_d = i32(lens)
    torch.cuda.synchronize()
    a = step(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = step(st)
    st.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attention(a[0], a[1], S_q(r, x, w, pos, hq), kc, vc, 0.1, np.arange(B + 1), lens, table, None, "bf16")


def S_q(r, x, w, pos, hq):
    q = torch.empty((x.shape[0], hq, x.shape[2]), dtype=x.dtype, device="cuda")
    E.emb_qk_norm_rotary(r.handle, pos, x[:, :hq], q, None, None, w, None, 1e-6)
    torch.cuda.synchronize()
    return q


def test_a_whole_step_in_a_graph():
    # rotation, norm with its gradient, append and attention captured once, replayed with new inputs
    # and lengths, with eager work between the replays
    gen = torch.Generator().manual_seed(43)
    rng = np.random.default_rng(43)
    hk, hq, D, page, B, P = 2, 8, 64, 16, 5, 333
    cap = 64
    pages = -(-P // page) + B * (cap // page) + 2
    kc, vc = paged(gen, "bf16", pages, page, hk, D)
    both = page_table(rng, pages, page, [P] + [cap] * B, extra=0)
    pt, table = both[:1].contiguous(), both[1:, :cap // page].contiguous()
    cache, r = E.KVCache(kc, vc), E.Rotary(D)
    x = randn(gen, (B, hq + 2 * hk, D), "bf16")
    w = torch.ones(D, device="cuda")
    lens, pos = i32([1] * B), torch.zeros(B, dtype=torch.int64, device="cuda")
    go, pl = i32([0, B]), i32([P])
    q, out = torch.empty((B, hq, D), dtype=x.dtype, device="cuda"), torch.empty((B, hq, D), dtype=x.dtype, device="cuda")
    dq, dw = torch.empty_like(q), torch.empty(D, device="cuda")
    lse = torch.empty((B, hq), device="cuda")
    ws = torch.empty(E.emb_prefix_attention_workspace_bytes(cache.handle, B, hq, 1, pt.shape[1], table.shape[1]),
                     dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(E.emb_qk_norm_rotary_workspace_bytes(B, hq, 0, D), dtype=torch.uint8, device="cuda")

    def step():
        E.emb_qk_norm_rotary(r.handle, pos, x[:, :hq], q, None, None, w, None, 1e-6)
        E.emb_kv_append(cache.handle, r.handle, x[:, hq:hq + hk], x[:, hq + hk:], None, lens, table, wk=w, eps=1e-6,
                        positions=pos)
        E.emb_prefix_attention(cache.handle, q, out, 0.125, None, lens, table, go, pl, pt, ws, lse=lse)
        E.emb_qk_norm_rotary_backward(r.handle, pos, x[:, :hq], out, dq, None, None, None, w, None, 1e-6, ws2, dw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(randn(gen, tuple(x.shape), "bf16"))
        lens.fill_(3 + 7 * i)
        pos.fill_(P + 2 + 7 * i)
        k0, v0 = kc.clone(), vc.clone()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, out, lse, dq, dw, kc, vc)]
        kc.copy_(k0), vc.copy_(v0)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (q, out, lse, dq, dw, kc, vc)):
            assert torch.equal(a, b), i
    cache.check_error()


def test_pages_beyond_32_bits():
    # a cache whose element offsets pass 2^32: the last pages of a 10 GiB pool
    hk, D, page = 1, 128, 64
    pages = (5 << 30) // (page * hk * D) + 5
    kc = torch.empty((pages, page, hk, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    assert kc.numel() > 1 << 32
    gen = torch.Generator().manual_seed(51)
    first = pages - 4
    kc[first:] = randn(gen, (4, page, hk, D), "bf16")
    vc[first:] = randn(gen, (4, page, hk, D), "bf16")
    cache = E.KVCache(kc, vc)
    table = i32([first + 1]).reshape(1, 1)
    pt = i32([first + 3, first]).reshape(1, 2)
    k, v = randn(gen, (1, hk, D), "bf16"), randn(gen, (1, hk, D), "bf16")
    E.emb_kv_append(cache.handle, None, k, v, None, i32([10]), table)
    q = randn(gen, (1, 2, D), "bf16")
    out, lse = run_attention(cache, q, 0.1, None, i32([10]), table, (i32([0, 1]), i32([100]), pt))
    cache.check_error()
    assert torch.equal(kc[first + 1, 9], k[0])
    shift = lambda t: t - first
    check_attention(out, lse, q, kc[first:], vc[first:], 0.1, [0, 1], [10], shift(table),
                    (i32([0, 1]), i32([100]), shift(pt)), "bf16")


# ---- attention: blocks that take several groups', sequences' and parts' work --------------

def test_attention_many_groups_and_empty_sequences():
    # more groups than a wave has lanes, runs of more sequences without tokens than that between two
    # with some, groups of such sequences alone, groups without sequences
    rng = np.random.default_rng(61)
    counts = []
    for i in range(12):
        counts += [int(n) for n in rng.integers(1, 6, 3)] + [0] * int(rng.choice([0, 1, 70, 130]))
    cuts = np.sort(rng.choice(len(counts) + 1, 79, replace=True))
    sizes = np.diff(np.concatenate([[0], cuts, [len(counts)]]))
    lens = [c + int(n) if c else int(n) for c, n in zip(counts, rng.integers(0, 40, len(counts)))]
    prefix = [int(n) for n in rng.integers(0, 50, len(sizes))]
    for hq, hk in ((4, 2), (2, 2)):
        q, kc, vc, off, lens_, table, groups = attention_case("bf16", 64, hq, hk, 16, counts, lens, sizes, prefix)
        cache = E.KVCache(kc, vc)
        out, lse = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
        cache.check_error()
        check_attention(out, lse, q, kc, vc, 0.125, off, lens, table, groups, "bf16")
        # the same sequences without prefixes
        out, lse = run_attention(cache, q, 0.125, i32(off), i32(lens), table)
        cache.check_error()
        check_attention(out, lse, q, kc, vc, 0.125, off, lens, table, None, "bf16")
        # in one group: a long run of empty sequences inside a tile of rows
        one = (i32([0, len(counts)]), groups[1][:1].contiguous(), groups[2][:1].contiguous())
        out, lse = run_attention(cache, q, 0.125, i32(off), i32(lens), table, one)
        cache.check_error()
        check_attention(out, lse, q, kc, vc, 0.125, off, lens, table, one, "bf16")


# (counts, lens, group sizes, prefixes, pages of table width to add): rows enough for tiles of 128 with the
# own slots taken along, parts of a prefix with them, own slots in blocks of their own (a wide table)
SHARED = {
    "tiles": ([1, 2] * 60, [20] * 60 + [33] * 60, [70, 50], [40, 333], 0),
    "parts": ([1, 3] * 40, [5, 40] * 40, [80], [1500], 0),
    "wide_table": ([1, 2] * 60, [20] * 60 + [33] * 60, [70, 50], [40, 333], 30),
    "no_prefix": ([1, 2] * 20, [20] * 20 + [33] * 20, [], [], 0),
}


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 96)])
@pytest.mark.parametrize("kind", list(SHARED))
def test_attention_rows_do_not_touch_each_other(dt, D, kind):
    counts, lens, gs, prefix, more = SHARED[kind]
    q, kc, vc, off, lens, table, groups = attention_case(dt, D, 4, 2, 16, counts, lens, gs, prefix)
    table = torch.cat([table, torch.full((len(lens), more), -1, dtype=torch.int32, device="cuda")], 1)
    cache = E.KVCache(kc, vc)
    base, base_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
    cache.check_error()
    check_attention(base, base_l, q, kc, vc, 0.125, off, lens, table, groups, dt)
    # sequence 7's own slots hold infinities, NaN and huge keys: only its rows may notice
    own = [int(x) for x in table[7][:-(-lens[7] // 16)]]
    t0, t1 = int(off[7]), int(off[8])
    rest = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    rest[t0:t1] = False
    k1, v1 = kc.clone(), vc.clone()
    for poison in (float("nan"), float("inf"), torch.finfo(DT[dt]).max):
        kc[own], vc[own] = poison, poison
        got, got_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
        assert torch.equal(got[rest], base[rest]) and torch.equal(got_l[rest], base_l[rest]), poison
        kc.copy_(k1), vc.copy_(v1)
    # an infinite value that only its last query sees: that row alone changes, and to an infinity
    if counts[7] > 1:
        pg, sl = int(table[7][(lens[7] - 1) // 16]), (lens[7] - 1) % 16
        vc[pg, sl] = float("inf")
        got, got_l = run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups)
        rest[t0:t1 - 1] = True
        assert torch.equal(got[rest], base[rest]) and torch.equal(got_l, base_l)
        assert torch.isposinf(got[t1 - 1]).all()
        vc.copy_(v1)
    # and its length is its own matter too
    other = list(lens)
    other[7] = counts[7]
    got, got_l = run_attention(cache, q, 0.125, i32(off), i32(other), table, groups)
    rest[t0:t1] = False
    assert torch.equal(got[rest], base[rest]) and torch.equal(got_l[rest], base_l[rest])


def test_attention_direct_result_in_strides_and_order_of_groups():
    # one part: the result is written by the prefix' blocks; the groups' order is not the lengths'
    case = ("bf16", 128, 8, 2, 16, [2] * 90, [7] * 90, [20, 50, 20], [100, 20, 240])
    q, kc, vc, off, lens, table, groups = attention_case(*case)
    cache = E.KVCache(kc, vc)
    out = torch.full((180, 8, 256), 5.0, dtype=q.dtype, device="cuda")
    got, lse = run_attention(cache, q, -0.3, i32(off), i32(lens), table, groups, out=out[..., 128:])
    cache.check_error()
    check_attention(got, lse, q, kc, vc, -0.3, off, lens, table, groups, "bf16")
    assert (out[..., :128] == 5.0).all()
