"""GPU tests of the attention of histories, its gradient and its step over a paged cache against their 64-bit
definitions (oracle/history_oracle.py).

Tolerances follow from the arithmetic, with u = 2^-24 (half an fp32 step) and h = eps / 2 of the heads' type:
  - a score is a sum of D products, a product and a sum: e = (D + 8) u max scale |q|.|k| + 8 u max |bias| absolute,
    which moves probabilities by that much relative;
  - out: probabilities are rounded to the heads' type (h) for the product with V: (h + 2 e + 128 u) sum p |v| and h |out|;
    lse: e + 256 u + 4 u |lse|;
  - gradients: P is off by 2 e + 300 u relative (score and lse), dP by (D + 8) u |dout|.|v|, sums by the number of
    their terms in a lane's chain and over the lanes (less than 300 u here); with |.| the same sums over magnitudes
    (of dS: P (|dP| + sum P |dP|)): dbias, in fp32 throughout: (2 e + (D + 600) u) |dbias|; dk, dv, whose factors
    are rounded: (h + 2 e + (D + 600) u) |.| and h of the result; dq besides is made from a row's sum that starts
    from the rounded out: what out may be off by, against |dout|, times scale sum P |k|.
"""
import gc

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from oracle import history_oracle as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


@pytest.fixture(autouse=True)
def _free_gpu():
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half(dt):
    return torch.finfo(DT[dt]).eps / 2


def close(got, want, err, dt, what):
    got = n64(got)
    tol = err + (half(dt) if dt != "f32" else U) * np.abs(want) * (1 + 1e-3) + TINY[dt]
    bad = ~((np.abs(got - want) <= tol) | (got == want))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {tol[i]}, worst {np.nanmax(np.abs(got - want) / tol)} times it")


class Call:
    """A batch of histories with its operands, and the library's calls on it."""

    def __init__(self, dt, dim, hq, hk, lens, causal=True, spec=None, memory="fused", seed=0, size=1.0):
        gen = torch.Generator().manual_seed(seed + dim + 7 * sum(lens))
        self.dt, self.dim, self.hq, self.hk, self.causal, self.spec = dt, dim, hq, hk, causal, spec
        self.T = T = sum(lens)
        self.off = [0]
        for n in lens:
            self.off.append(self.off[-1] + n)
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        n = spec[0] if spec else 0
        self.h = E.HistoryAttention(hq, hk, dim, dt, causal=causal, buckets=n, exact=spec[1] if spec else 0,
                                    far=spec[2] if spec else 0)
        self.scale = float(np.float32(dim ** -0.5))

        def new(heads, fill=True):
            x = (size * torch.randn((T, heads, dim), generator=gen)).to(DT[dt])
            if memory == "heads_first":
                y = torch.empty((heads, max(T, 1), dim), dtype=DT[dt], device="cuda").transpose(0, 1)[:T]
            elif memory == "wide":      # rows and heads apart
                y = torch.full((max(T, 1), heads + 1, dim + 16), float("nan"), dtype=DT[dt], device="cuda")[:T, :heads, 8:8 + dim]
            else:
                y = torch.empty((T, heads, dim), dtype=DT[dt], device="cuda")
            y.copy_(x)
            return y
        if memory == "fused":
            fused = (size * torch.randn((T, hq + 2 * hk, dim), generator=gen)).to(DT[dt]).cuda()
            self.q, self.k, self.v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
        else:
            self.q, self.k, self.v = new(hq), new(hk), new(hk)
        self.dout = new(hq)
        self.bias = torch.randn((self.h.bias_rows, hq), generator=gen).cuda() if spec else None
        self.out, self.dq, self.dk, self.dv = new(hq), new(hq), new(hk), new(hk)
        self.lse = torch.full((T, hq), 7.0, device="cuda")
        self.dbias = torch.full_like(self.bias, 7.0) if spec else None
        self.ws = torch.full((E.emb_history_attention_workspace_bytes(self.h.handle, T, len(lens)) or 16,), 0x7f,
                             dtype=torch.uint8, device="cuda")

    def forward(self, **kw):
        E.emb_history_attention(self.h.handle, self.q, self.k, self.v, self.out, self.offsets, bias=self.bias,
                                lse=self.lse, **kw)
        return self.out, self.lse

    def backward(self, **kw):
        E.emb_history_attention_backward(self.h.handle, self.q, self.k, self.v, self.out, self.lse, self.dout, self.dq,
                                         self.dk, self.dv, self.offsets, self.ws, bias=self.bias, dbias=self.dbias, **kw)
        return [t for t in (self.dq, self.dk, self.dv, self.dbias) if t is not None]

    def arrays(self):
        return n64(self.q), n64(self.k), n64(self.v)

    def score_error(self):
        q, k, _ = self.arrays()
        if not self.T:
            return 0.0
        big = self.scale * np.abs(q).sum(2).max() * np.abs(k).max()
        norm = self.scale * np.sqrt((q ** 2).sum(2).max() * (k ** 2).sum(2).max())
        b = 0.0 if self.bias is None else np.abs(n64(self.bias)[n64(self.bias) > H.HIDDEN]).max(initial=0.0)
        return (self.dim + 8) * U * min(big, norm) + 8 * U * b

    def check_forward(self):
        q, k, v = self.arrays()
        want, lse, mag = H.attention(q, k, v, self.off, self.scale, self.causal, n64(self.bias), self.spec)
        e = self.score_error()
        self.tol_out = (half(self.dt) + 2 * e + 128 * U) * mag + half(self.dt) * np.abs(want)
        close(self.out, want, self.tol_out, self.dt, "out")
        close(self.lse, lse, e + 256 * U + 4 * U * np.abs(np.where(np.isinf(lse), 0, lse)), "f32", "lse")

    def check_backward(self):
        q, k, v = self.arrays()
        do = n64(self.dout)
        g = H.attention_backward(q, k, v, do, self.off, self.scale, self.causal, n64(self.bias), self.spec)
        rel = 2 * self.score_error() + (self.dim + 600) * U
        for n, t in (("dk", self.dk), ("dv", self.dv)):
            close(t, g[n], (half(self.dt) + rel) * g[f"|{n}|"], self.dt, n)
        # scale sum P |k| of each row
        pk = H.attention(q, k, np.abs(k), self.off, self.scale, self.causal, n64(self.bias), self.spec)[0] * self.scale
        slip = (np.abs(do) * self.tol_out).sum(2, keepdims=True)
        close(self.dq, g["dq"], (half(self.dt) + rel) * g["|dq|"] + slip * pk, self.dt, "dq")
        if self.spec:
            close(self.dbias, g["dbias"], rel * g["|dbias|"], "f32", "dbias")


SPEC = (32, 16, 128)
CASES = [
    # dtype, dim, q heads, k heads, lengths, causal, (buckets, exact, far), memory
    ("bf16", 64, 4, 2, [5], True, None, "fused"),
    ("f16", 64, 2, 2, [1], True, (8, 4, 20), "fused"),
    ("bf16", 128, 2, 1, [32], True, SPEC, "plain"),
    ("bf16", 128, 1, 1, [33], False, SPEC, "plain"),
    ("f16", 128, 4, 4, [64, 31], True, SPEC, "wide"),
    ("bf16", 96, 4, 2, [65, 0, 1, 127], True, SPEC, "heads_first"),
    ("f16", 96, 3, 1, [0, 128, 0], False, (16, 8, 64), "fused"),
    ("bf16", 64, 8, 1, [129, 2, 63], True, (64, 32, 1024), "fused"),
    ("f16", 64, 2, 1, [200, 300], False, (8, 8, 0), "wide"),
    ("bf16", 128, 6, 2, [300, 17], True, (5, 1, 9), "fused"),
    ("f16", 128, 2, 2, [257], True, (128, 1, 1 << 30), "plain"),
    ("bf16", 96, 2, 1, [260], False, None, "heads_first"),
    ("f16", 64, 2, 2, [1] * 70 + [40], True, (10, 3, 5), "fused"),
    ("bf16", 64, 1, 1, [700], True, (12, 4, 60), "plain"),
    ("bf16", 64, 1, 1, [500], False, (12, 4, 60), "plain"),
    ("f16", 128, 1, 1, [400], True, (1, 1, 0), "fused"),
]


@pytest.mark.parametrize("dt,dim,hq,hk,lens,causal,spec,memory", CASES)
def test_attention_and_gradient(dt, dim, hq, hk, lens, causal, spec, memory):
    c = Call(dt, dim, hq, hk, lens, causal, spec, memory)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.h.check_error()
    # again: the same bits, also where the bias' gradient is not wanted
    first = [t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv)]
    dbias, c.dbias = c.dbias, None
    for t in (c.dq, c.dk, c.dv):
        t.fill_(3)
    c.forward()
    c.backward()
    assert all(torch.equal(a, b) for a, b in zip(first, (c.out, c.lse, c.dq, c.dk, c.dv)))
    if spec:
        c.dbias = torch.zeros_like(dbias)
        c.backward()
        assert torch.equal(c.dbias, dbias)
    if memory == "wide":       # nothing beside the heads was written
        for t in (c.out, c.dq, c.dk, c.dv):
            rest = t._base.clone()
            rest[:c.T, :t.shape[1], 8:8 + dim] = float("nan")
            assert rest.isnan().all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_sequence_does_not_depend_on_its_neighbours(dt):
    """Neither their length nor what they hold changes a bit of a sequence's results."""
    a = Call(dt, 64, 4, 2, [40, 150, 33], True, SPEC)
    b = Call(dt, 64, 4, 2, [150], True, SPEC)
    for x, y in ((a.q, b.q), (a.k, b.k), (a.v, b.v), (a.dout, b.dout)):
        y.copy_(x[40:190])
        x[:40] = float("nan")
        x[190:] = float("inf")
    b.bias.copy_(a.bias)
    a.forward(), b.forward(), a.backward(), b.backward()
    for x, y in ((a.out, b.out), (a.lse, b.lse), (a.dq, b.dq), (a.dk, b.dk), (a.dv, b.dv)):
        assert torch.equal(x[40:190], y) and not y.isnan().any()


@pytest.mark.parametrize("dt,dim", [("bf16", 64), ("f16", 96), ("bf16", 128), ("f16", 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_later_items_have_no_influence(dt, dim, bad):
    """A value that is no number, at one place: rows before it are what they are without it."""
    n, at = 150, 77
    a, b = (Call(dt, dim, 2, 1, [n], True, SPEC, "plain") for _ in range(2))
    for t in (a.k, a.v):
        t[at, 0, 5] = bad
    a.forward(), b.forward()
    assert torch.equal(a.out[:at], b.out[:at]) and torch.equal(a.lse[:at], b.lse[:at])
    assert not a.out[at:].isfinite().all()
    a.out.copy_(b.out), a.lse.copy_(b.lse)
    a.backward(), b.backward()
    assert torch.equal(a.dq[:at], b.dq[:at])
    # the gradients of keys behind the place see only queries behind it; those of keys up to it are its own
    c = Call(dt, dim, 2, 1, [n], True, SPEC, "plain")
    for t in (c.q, c.dout):
        t[at, 1, 3] = bad
    c.out.copy_(b.out), c.lse.copy_(b.lse)
    c.backward()
    assert torch.equal(c.dk[at + 1:], b.dk[at + 1:]) and torch.equal(c.dv[at + 1:], b.dv[at + 1:])
    assert torch.equal(c.dq[:at], b.dq[:at]) and torch.equal(c.dq[:, 0], b.dq[:, 0])


@pytest.mark.parametrize("lowest", [float("-inf"), torch.finfo(torch.float32).min, -2.0 ** 100])
@pytest.mark.parametrize("dt,causal", [("bf16", True), ("f16", False)])
def test_hidden_distances(dt, causal, lowest):
    """Entries that hide; rows that see nothing are zeros, -inf, and have no gradient."""
    c = Call(dt, 64, 2, 1, [70, 3], causal, (16, 8, 30), "plain")
    c.bias[0] = lowest
    c.bias[10:14, 0] = lowest
    if not causal:
        c.bias[16:, 1] = lowest
    c.forward()
    c.check_forward()
    empty = torch.isneginf(c.lse)
    assert empty[0].any() and (c.out[empty] == 0).all()
    c.backward()
    c.check_backward()
    assert (c.dq[empty] == 0).all() and (c.dbias[0] == 0).all()
    c.bias.fill_(lowest)
    c.forward(), c.backward()
    assert (c.out == 0).all() and torch.isneginf(c.lse).all()
    assert all((t == 0).all() for t in (c.dq, c.dk, c.dv, c.dbias))


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_small_and_large_values(size):
    """Sizes of operands at which fp16 score gradients would underflow, and one-sided softmaxes."""
    c = Call("f16", 64, 2, 1, [300], True, SPEC, "plain", size=min(size, 6.0))
    c.dout.mul_(size)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


def test_gradient_against_differences():
    """The library's gradient against differences of the 64-bit definition."""
    c = Call("f16", 64, 2, 1, [30], True, (8, 4, 16), "plain")
    c.forward(), c.backward()
    q, k, v = c.arrays()
    do, bias = n64(c.dout), n64(c.bias)
    rng = np.random.default_rng(0)

    def loss(q, k, v, bias):
        return (H.attention(q, k, v, c.off, c.scale, True, bias, c.spec)[0] * do).sum()
    for i, got in enumerate((c.dq, c.dk, c.dv, c.dbias)):
        args = [q, k, v, bias]
        d = rng.normal(size=args[i].shape)
        d /= np.linalg.norm(d)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        slope = (loss(*hi) - loss(*lo)) / 2e-5
        # a unit direction: off by at most the norm of what each element may be off by
        tol = 2 * (half("f16") + 2 * c.score_error() + 700 * U) * np.linalg.norm(n64(got)) * 3 + 1e-6
        assert abs((n64(got) * d).sum() - slope) <= tol


def test_no_tokens():
    c = Call("bf16", 64, 2, 1, [0, 0], True, SPEC)
    c.forward()
    c.backward()
    assert (c.dbias == 0).all()


def test_row_sums_of_the_bias_gradient_cancel():
    """dS sums to zero along each row, so dbias to zero over its rows, up to fp32's rounding."""
    for dt in ("bf16", "f16"):
        c = Call(dt, 128, 4, 2, [1500, 700], True, (64, 32, 1024))
        c.forward(), c.backward()
        mag = np.abs(n64(c.dbias)).sum(0)
        assert (np.abs(n64(c.dbias).sum(0)) <= 2e-4 * mag).all()


@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [5, 50, 60, 100], [0, 10, 20, 90], [-7, 10, 20, 1 << 30]])
def test_offsets_that_break_their_contract_are_reported(offsets):
    c = Call("bf16", 64, 2, 1, [50, 10, 40], True, SPEC, "wide")
    c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    c.forward()
    with pytest.raises(E.EmbError) as e:
        c.h.check_error()
    assert e.value.code == E.EMB_E_INVAL
    c.h.check_error()           # cleared
    c.backward()
    with pytest.raises(E.EmbError):
        c.h.check_error()
    for t in (c.out, c.dq, c.dk, c.dv):
        rest = t._base.clone()
        rest[:c.T, :t.shape[1], 8:8 + 64] = float("nan")
        assert rest.isnan().all()


def test_graph_and_streams():
    a, b = (Call("bf16", 128, 4, 2, [300, 77], True, SPEC, seed=s) for s in (1, 2))
    ref = []
    for c in (a, b):
        c.forward(), c.backward()
        ref.append([t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv, c.dbias)])
    torch.cuda.synchronize()
    # two calls at once, with a workspace each
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for c, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                c.forward(), c.backward()
    torch.cuda.synchronize()
    for c, r in zip((a, b), ref):
        assert all(torch.equal(x, y) for x, y in zip((c.out, c.lse, c.dq, c.dk, c.dv, c.dbias), r))
    # on another stream than the current one
    a.out.zero_()
    torch.cuda.synchronize()
    a.forward(stream=s1)
    s1.synchronize()
    assert torch.equal(a.out, ref[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward(), a.backward()
    for i in range(4):
        a.q.mul_(1.25), a.dout.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (a.out, a.lse, a.dq, a.dk, a.dv, a.dbias)]
        a.forward(), a.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (a.out, a.lse, a.dq, a.dk, a.dv, a.dbias)))


def test_strides_beyond_32_bits():
    """Tokens whose elements lie past 2^32 bytes."""
    n, ts = 300, 1 << 23
    c = Call("bf16", 64, 1, 1, [n], True, SPEC, "plain")
    base = torch.empty(n * ts, dtype=torch.bfloat16, device="cuda")
    far = [base.as_strided((n, 1, 64), (ts, 64, 1), 64 * i) for i in range(8)]
    c.forward(), c.backward()
    want = [t.clone() for t in (c.out, c.dq, c.dk, c.dv, c.dbias)]
    for x, t in zip(far, (c.q, c.k, c.v, c.dout)):
        x.copy_(t)
    c.q, c.k, c.v, c.dout, c.out, c.dq, c.dk, c.dv = far
    c.forward(), c.backward()
    assert all(torch.equal(x, y) for x, y in zip(want, (c.out, c.dq, c.dk, c.dv, c.dbias)))


# ---- one new item of each history ------------------------------------------------

class Step:
    def __init__(self, dt, dim, hq, hk, lens, page, spec=None, width=0, seed=0, heads_first=True):
        gen = torch.Generator().manual_seed(seed + 3 * dim + sum(lens))
        self.dt, self.dim, self.spec, self.lens_list = dt, dim, spec, lens
        B = len(lens)
        need = [-(-n // page) for n in lens]
        pool = torch.randperm(sum(need) + 3, generator=gen).to(torch.int32)
        width = max([width, 1] + need)
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = pool[at:at + n]
            at += n
        shape = (pool.numel(), hk, page, dim) if heads_first else (pool.numel(), page, hk, dim)
        kc, vc = ((torch.randn(shape, generator=gen)).to(DT[dt]).cuda() for _ in range(2))
        self.kc, self.vc = (t.transpose(1, 2) if heads_first else t for t in (kc, vc))
        self.cache = E.KVCache(self.kc, self.vc)
        self.h = E.HistoryAttention(hq, hk, dim, dt, buckets=spec[0] if spec else 0, exact=spec[1] if spec else 0,
                                    far=spec[2] if spec else 0)
        self.scale = float(np.float32(dim ** -0.5))
        self.q = torch.randn((B, hq, dim), generator=gen).to(DT[dt]).cuda()
        self.bias = torch.randn((self.h.bias_rows, hq), generator=gen).cuda() if spec else None
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.out, self.lse = torch.full_like(self.q, 7.0), torch.full((B, hq), 7.0, device="cuda")
        self.ws = torch.full((E.emb_history_step_workspace_bytes(self.h.handle, self.cache.handle, B, width),), 0x7f,
                             dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        E.emb_history_step(self.h.handle, self.cache.handle, self.q, self.out, self.lens, self.table, self.ws,
                           bias=self.bias, lse=self.lse, **kw)

    def check(self):
        q, kc, vc = n64(self.q), n64(self.kc), n64(self.vc)
        want, lse, mag = H.step(q, kc, vc, self.lens_list, self.table.cpu().numpy(), self.scale, n64(self.bias), self.spec)
        k2 = np.nan_to_num(kc)
        e = (self.dim + 8) * U * self.scale * np.sqrt((q ** 2).sum(2).max() * (k2 ** 2).sum(3).max()) + \
            (8 * U * np.abs(n64(self.bias)[n64(self.bias) > H.HIDDEN]).max(initial=0.0) if self.spec else 0.0)
        close(self.out, want, (half(self.dt) + 2 * e + 128 * U) * mag + half(self.dt) * np.abs(want), self.dt, "out")
        close(self.lse, lse, e + 256 * U + 4 * U * np.abs(np.where(np.isinf(lse), 0, lse)), "f32", "lse")


@pytest.mark.parametrize("dt,dim,hq,hk,lens,page,spec,width,heads_first", [
    ("bf16", 64, 4, 2, [1], 16, None, 0, True),
    ("f16", 128, 8, 2, [33, 0, 64, 1], 16, SPEC, 0, True),
    ("bf16", 128, 4, 4, [300, 257], 32, SPEC, 0, False),
    ("f16", 96, 6, 2, [129, 700], 7, (16, 8, 64), 0, True),
    ("bf16", 96, 32, 1, [95], 1, (8, 8, 0), 0, True),
    ("f16", 64, 5, 1, [2000], 64, (64, 32, 1024), 0, True),
    ("bf16", 64, 2, 2, [31, 40], 16, (64, 1, 1 << 30), 200, True),      # a table wider than needed: empty parts
    ("bf16", 128, 2, 1, [5000], 128, (20, 4, 700), 0, True),
    ("f16", 64, 1, 1, [17000], 16, None, 0, False),
])
def test_step(dt, dim, hq, hk, lens, page, spec, width, heads_first):
    s = Step(dt, dim, hq, hk, lens, page, spec, width, heads_first=heads_first)
    s.run()
    s.check()
    s.cache.check_error()
    first = [s.out.clone(), s.lse.clone()]
    s.run()
    assert torch.equal(first[0], s.out) and torch.equal(first[1], s.lse)
    lse, s.lse = s.lse, None
    s.out.zero_()
    s.run()
    assert torch.equal(first[0], s.out)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_step_sees_its_slots_only(dt):
    """What lies behind a history's last slot, in its last page and elsewhere, changes no bit."""
    a, b = (Step(dt, 64, 4, 2, [45, 300, 7], 16, SPEC) for _ in range(2))
    used = torch.zeros(a.kc.shape[:2], dtype=torch.bool, device="cuda")
    for r, n in enumerate(a.lens_list):
        for j in range(n):
            used[a.table[r, j // 16], j % 16] = True
    for t in (a.kc, a.vc):
        t[~used] = float("nan")
    a.run(), b.run()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and not a.out.isnan().any()


def test_step_hidden_and_empty():
    s = Step("bf16", 64, 2, 1, [0, 40, 1], 16, (8, 4, 16))
    s.bias[0] = float("-inf")
    s.run()
    s.check()
    assert (s.out[0] == 0).all() and (s.out[2] == 0).all() and torch.isneginf(s.lse[2]).all()


def test_step_reports_bad_pages_and_lengths():
    for what in ("page", "long", "negative"):
        s = Step("f16", 64, 2, 1, [300, 20], 16, SPEC)
        good = Step("f16", 64, 2, 1, [300, 20], 16, SPEC)
        if what == "page":
            s.table[1, 0] = 1 << 30
        else:
            s.lens[1] = 1 << 29 if what == "long" else -5
            if what == "long":
                s.table[1] = s.table[0]
        s.run(), good.run()
        with pytest.raises(E.EmbError) as e:
            s.cache.check_error()
        assert e.value.code == E.EMB_E_BOUNDS
        assert torch.equal(s.out[0], good.out[0])
        if what == "negative":
            assert (s.out[1] == 0).all()


def test_step_is_the_last_row_of_the_attention():
    c = Call("bf16", 128, 4, 2, [200], True, SPEC, "plain")
    s = Step("bf16", 128, 4, 2, [200], 16, SPEC)
    s.bias.copy_(c.bias)
    s.q.copy_(c.q[-1:])
    for j in range(200):
        p = int(s.table[0, j // 16])
        s.kc[p, j % 16], s.vc[p, j % 16] = c.k[j], c.v[j]
    c.forward()
    s.run()
    s.check()
    # both round probabilities and the result
    tol = 4 * half("bf16") * n64(c.v[:200]).__abs__().max()
    assert np.abs(n64(s.out[0]) - n64(c.out[-1])).max() <= tol


def test_step_in_a_graph_on_other_streams():
    s = Step("bf16", 64, 4, 2, [700, 90], 16, SPEC)
    graph = torch.cuda.CUDAGraph()
    s.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(3):
        s.q.mul_(-1.5)
        s.lens.sub_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = s.out.clone()
        s.run(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert torch.equal(got, s.out)


def test_nearly_as_many_sequences_as_a_launch_takes():
    """A million sequences, three of which have tokens: the bits of those three alone."""
    lens, at, n = [50, 1, 130], [5, 777_777, 1_040_000], 1_045_000
    a = Call("bf16", 64, 16, 16, lens)
    where = torch.zeros(n, dtype=torch.int32)
    where[at] = torch.tensor(lens, dtype=torch.int32)
    many = torch.cat([torch.zeros(1, dtype=torch.int32), where.cumsum(0).to(torch.int32)]).cuda()
    assert (n + sum(lens) // 64) * 16 < 1 << 24 <= (n + 5000) * 16
    a.forward()
    want = [t.clone() for t in [a.out, a.lse] + a.backward()]
    a.offsets = many
    a.ws = torch.empty(E.emb_history_attention_workspace_bytes(a.h.handle, a.T, n), dtype=torch.uint8, device="cuda")
    for t in (a.out, a.lse, a.dq, a.dk, a.dv):
        t.fill_(3)
    a.forward()
    assert all(torch.equal(x, y) for x, y in zip(want, [a.out, a.lse] + a.backward()))
    a.h.check_error()


@pytest.mark.parametrize("dt,dim", [("bf16", 64), ("f16", 64), ("bf16", 96), ("f16", 96), ("bf16", 128), ("f16", 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("spec", [SPEC, None])
def test_one_key_has_no_gradient_of_scores(dt, dim, causal, spec):
    """A softmax over one key is constant: zero gradients of queries, keys and biases, exactly; also of the first
    rows of longer causal histories."""
    c = Call(dt, dim, 4, 2, [1] * 37, causal, spec)
    c.forward()
    c.backward()
    assert not c.dq.any() and not c.dk.any() and (spec is None or not c.dbias.any())
    c.check_forward()
    c.check_backward()
    if causal:
        c = Call(dt, dim, 4, 2, [70, 3], causal, spec)
        c.forward()
        c.backward()
        assert not c.dq[0].any() and not c.dq[70].any() and c.dq[1].any()
        c.check_forward()
        c.check_backward()
