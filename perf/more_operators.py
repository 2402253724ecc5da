"""Timed cases of what trains and serves a layer over users' histories: layer
norm and its gradient, dropout with a residual sum, the attention of a ragged
batch of histories over themselves with a learned bias by relative position and
its gradient, and the attention of one new token of each history over a paged
cache with the same bias.

With ``own`` false, ``run`` computes each operator from elementary torch
operations in 32 bits (sums over many rows in 64); with ``own`` true it calls
the library. ``exact`` computes the same outputs in 64 bits from the
definitions. Heads, lengths and dimensions are generic.
"""
from __future__ import annotations

import math
import random
from fractions import Fraction

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # activations of a few serving requests: what counts is the latency of the call
        dict(name="norm_few", op="norm", dtype="bf16", out="bf16", rows=48, dim=512, bias=True),
        # embedding rows of a training batch (fp32), normed for a 16-bit projection
        dict(name="norm_rows", op="norm", dtype="f32", out="bf16", rows=262144, dim=128, bias=True),
        # gradient of a wide layer's norm with those of its weights, odd number of rows
        dict(name="norm_back", op="norm_back", dtype="bf16", out="bf16", rows=24577, dim=1024, bias=True),
        # dropout of a small batch's fp32 rows of odd width, no residual
        dict(name="drop_few", op="drop", dtype="f32", rows=509, dim=65, p=0.1, residual=False),
        # dropout of a layer's output and the sum with its input
        dict(name="drop_add", op="drop", dtype="bf16", rows=32768, dim=1024, p=0.2, residual=True),
        # one user's short history: latency
        dict(name="attend_few", op="attend", dtype="bf16", seqs=1, tokens=50, hq=8, hk=2, dim=64, causal=True,
             buckets=32, ragged=1),
        # a training batch of short histories, both directions, a key head of its own for each query head
        dict(name="attend_users", op="attend", dtype="f16", seqs=256, tokens=51201, hq=8, hk=8, dim=64, causal=False,
             buckets=32, ragged=2),
        # few long histories, shared key heads: bound by the matrix products
        dict(name="attend_long", op="attend", dtype="bf16", seqs=3, tokens=24577, hq=16, hk=4, dim=128, causal=True,
             buckets=64, ragged=3),
        # gradient of a training batch of histories, shared key heads
        dict(name="attend_back_users", op="attend_back", dtype="bf16", seqs=128, tokens=40001, hq=8, hk=2, dim=64,
             causal=True, buckets=32, ragged=4),
        # gradient of few long histories
        dict(name="attend_back_long", op="attend_back", dtype="f16", seqs=3, tokens=12289, hq=16, hk=4, dim=128,
             causal=True, buckets=64, ragged=5),
        # the newest item of each user of a serving batch
        dict(name="step_users", op="step", dtype="bf16", seqs=61, hq=32, hk=8, dim=128, page=16, held=3000,
             buckets=32, ragged=6),
        # one user with a very long history
        dict(name="step_long", op="step", dtype="f16", seqs=1, hq=16, hk=4, dim=64, page=32, held=60001,
             buckets=64, ragged=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "drop", "attend", "attend_back", "step"])
    if op in ("norm", "norm_back", "drop"):
        dim = rng.choice([64, 128, 256, 512, 1024, _log_int(rng, 3, 2000)])
        rows = _log_int(rng, 1, min(262144, (1 << 25) // dim))
        c = dict(op=op, rows=rows, dim=dim, dtype=rng.choice(["bf16", "f16", "f32"]))
        if op == "drop":
            c.update(p=rng.uniform(0.01, 0.6), residual=rng.random() < 0.5)
        else:
            c.update(out=rng.choice([c["dtype"], "bf16", "f16"]) if c["dtype"] == "f32" else c["dtype"],
                     bias=rng.random() < 0.7)
        return c
    hk = rng.choice([1, 2, 4])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), hk=hk, hq=hk * rng.choice([1, 2, 4]),
             dim=rng.choice([64, 96, 128]), buckets=rng.choice([0, 16, 32, 64]), ragged=rng.randrange(1 << 30))
    if op == "step":
        c.update(seqs=_log_int(rng, 1, 64), page=rng.choice([16, 32, 64]))
        c["held"] = _log_int(rng, 1, 65536 // c["seqs"])
        return c
    c.update(tokens=_log_int(rng, 1, 24577), causal=rng.random() < 0.6)
    c["seqs"] = min(c["tokens"], _log_int(rng, 1, 256))
    largest = max(work(x)["flops"] for x in listed())
    while work(c)["flops"] > largest:
        c["tokens"] = c["tokens"] * 2 // 3
    c["seqs"] = min(c["seqs"], c["tokens"])
    return c


# ---- sizes that follow from a case -------------------------------------------

def _lengths(case):
    """Lengths of the histories, from the case alone."""
    r = random.Random(case["ragged"])
    if case["op"] == "step":
        if case["seqs"] == 1:
            return [case["held"]]
        return [r.randrange(1, case["held"] + 1) for _ in range(case["seqs"])]
    n, parts = case["tokens"], min(case["seqs"], case["tokens"])
    cuts = sorted(r.sample(range(1, n), parts - 1)) if parts > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [n])]


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_back"):
        n = case["rows"] * case["dim"]
        out = 4 if case["out"] == "f32" else 2
        if op == "norm":
            return {"bytes": n * (size + out), "flops": 8 * n}
        return {"bytes": n * (2 * size + out), "flops": 17 * n}
    if op == "drop":
        n = case["rows"] * case["dim"]
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 3 * n}
    lens = _lengths(case)
    hq, hk, D = case["hq"], case["hk"], case["dim"]
    if op == "step":
        return {"bytes": 2 * sum(lens) * hk * D * size + 2 * len(lens) * hq * D * size,
                "flops": 4 * sum(lens) * hq * D}
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    T = sum(lens)
    if op == "attend":
        return {"bytes": T * (2 * hq + 2 * hk) * D * size + 4 * T * hq, "flops": 4 * pairs * hq * D}
    return {"bytes": T * (4 * hq + 4 * hk) * D * size + 4 * T * hq, "flops": 10 * pairs * hq * D}


def _bias_shape(case):
    """Buckets of a direction, the distances with a bucket of their own, and where the last bucket starts."""
    b = case["buckets"]
    return b, b // 2, 16 * b


def _bias_rows(case):
    return case["buckets"] * (1 if case.get("causal", True) else 2)


def _starts(case):
    """First distance of each bucket: bucket k >= exact starts at the smallest integer that is at least
    exact * (far / exact) ** ((k - exact) / (buckets - exact))."""
    b, exact_, far = _bias_shape(case)
    first = list(range(exact_ + 1))
    n = b - exact_
    for k in range(1, n):
        d = int(exact_ * (far / exact_) ** (k / n)) - 1
        while Fraction(d, exact_) ** n < Fraction(far, exact_) ** k:
            d += 1
        first.append(d)
    return first[:b]


# ---- inputs ----------------------------------------------------------------------

def _heads(gen, tokens, heads, dim, dtype, dev):
    """Activations of a projection: heads of unlike size."""
    size = 0.5 + torch.rand((1, heads, 1), generator=gen, device=dev)
    return (torch.randn((tokens, heads, dim), generator=gen, device=dev) * size).to(dtype)


def _inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    op = case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if op in ("norm", "norm_back", "drop"):
        R, D = case["rows"], case["dim"]
        # rows of unlike size and mean
        x = randn(R, D) * (0.1 + 2 * torch.rand((R, 1), generator=gen, device=dev)) + 0.5 * randn(R, 1)
        s["x"] = x.to(dt)
        if op == "drop":
            s["r"] = randn(R, D).to(dt) if case["residual"] else None
            s["key"] = random.Random(seed).randrange(1 << 64)
            s["step"] = torch.tensor([random.Random(seed + 1).randrange(1 << 40)], dtype=torch.int64, device=dev)
            s["y"] = torch.empty((R, D), dtype=dt, device=dev)
            return s
        out = DTYPES[case["out"]]
        s["w"] = 1.0 + 0.2 * randn(D)
        s["b"] = 0.3 * randn(D) if case["bias"] else None
        s["eps"] = 1e-5
        if op == "norm":
            s["y"] = torch.empty((R, D), dtype=out, device=dev)
        else:
            s["dy"] = randn(R, D).to(out)
            s["dx"] = torch.empty((R, D), dtype=dt, device=dev)
        return s
    lens = _lengths(case)
    s["lens"] = lens
    hq, hk, D = case["hq"], case["hk"], case["dim"]
    s["scale"] = 1.0 / math.sqrt(D)
    s["bias"] = randn(_bias_rows(case), hq) if case["buckets"] else None
    if op == "step":
        B, page = case["seqs"], case["page"]
        need = [-(-n // page) for n in lens]
        pool = torch.randperm(sum(need) + 8, generator=gen, device=dev).to(torch.int32)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = pool[at:at + n]
            at += n
        s["table"] = table
        s["lens_dev"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        shape = (pool.numel(), hk, page, D)  # a page holds each head's rows together
        s["kc"] = randn(*shape).to(dt).transpose(1, 2)
        s["vc"] = randn(*shape).to(dt).transpose(1, 2)
        s["q"] = _heads(gen, B, hq, D, dt, dev)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, hq), dtype=torch.float32, device=dev)
        return s
    T = sum(lens)
    # q, k and v as slices of one projection's output
    fused = _heads(gen, T, hq + 2 * hk, D, dt, dev)
    s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    s["offsets"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    s["out"] = torch.empty((T, hq, D), dtype=dt, device=dev)
    s["lse"] = torch.empty((T, hq), dtype=torch.float32, device=dev)
    if op == "attend_back":
        s["dout"] = randn(T, hq, D).to(dt)
        s["dq"] = torch.empty((T, hq, D), dtype=dt, device=dev)
        s["dk"] = torch.empty((T, hk, D), dtype=dt, device=dev)
        s["dv"] = torch.empty((T, hk, D), dtype=dt, device=dev)
        s["dbias"] = None if s["bias"] is None else torch.empty_like(s["bias"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if "ragged" in case and case["buckets"]:
        s["starts"] = torch.tensor(_starts(case), device="cuda")
    if op == "attend_back":
        # what the forward pass of the step has left
        got = _plain_attend(s)
        s["out"], s["lse"] = got["out"], got["lse"]
    if own:
        from dlrm_sparse_embedding_amd import emb as E
        if op == "norm_back":
            n = E.emb_layer_norm_workspace_bytes(case["rows"], case["dim"])
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
            s["dw"] = torch.empty(case["dim"], device="cuda")
            s["db"] = torch.empty(case["dim"], device="cuda") if case["bias"] else None
        if "ragged" in case:
            buckets, exact_, far = _bias_shape(case)
            s["h"] = E.HistoryAttention(case["hq"], case["hk"], case["dim"], case["dtype"], scale=s["scale"],
                                        causal=case.get("causal", True), buckets=buckets, exact=exact_, far=far)
        if op == "attend_back":
            n = E.emb_history_attention_workspace_bytes(s["h"].handle, case["tokens"], len(s["lens"]))
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        if op == "step":
            s["cache"] = E.KVCache(s["kc"], s["vc"])
            n = E.emb_history_step_workspace_bytes(s["h"].handle, s["cache"].handle, case["seqs"],
                                                   s["table"].shape[1])
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms -------------------------------------------------------------------

def _plain_norm(s):
    x = s["x"].float()
    c = x - x.mean(-1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["w"]
    return {"y": (y if s["b"] is None else y + s["b"]).to(s["y"].dtype)}


def _plain_norm_back(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"])
    h = c * r
    g = dy * s["w"]
    dx = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    res = {"dx": dx.to(s["dx"].dtype), "dw": (dy * h).sum(0, dtype=torch.float64).float()}
    if s["b"] is not None:
        res["db"] = dy.sum(0, dtype=torch.float64).float()
    return res


def _random_words(rows, units, key, step, second):
    """Philox4x32-10 at (unit, row, step): four 32-bit words for each unit of 8 columns, int64 [rows, units, 4]."""
    dev = step.device
    m = 0xFFFFFFFF
    c = [torch.arange(units, device=dev)[None, :].expand(rows, units),
         torch.arange(rows, device=dev)[:, None].expand(rows, units),
         (step & m).expand(rows, units), ((step >> 32) & 0x7FFFFFFF | (second << 31)).expand(rows, units)]
    k0, k1 = key & m, key >> 32

    def wide(a, mul):
        low = (a & 0xFFFF) * mul
        return ((a >> 16) * mul + (low >> 16)) >> 16, (a * mul) & m

    for _ in range(10):
        h0, l0 = wide(c[0], 0xD2511F53)
        h1, l1 = wide(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return torch.stack(c, -1)


def _random_halves(rows, dim, key, step, second):
    w = _random_words(rows, -(-dim // 8), key, step, second)
    return torch.stack([w & 0xFFFF, w >> 16], -1).reshape(rows, -1)[:, :dim]


def _kept(s):
    case = s["case"]
    rows, dim = case["rows"], case["dim"]
    first = _random_halves(rows, dim, s["key"], s["step"], 0)
    second = _random_halves(rows, dim, s["key"], s["step"], 1)
    return (first << 16 | second) >= int(case["p"] * 2 ** 32 + 0.5)


def _plain_drop(s):
    x = s["x"].float()
    p = int(s["case"]["p"] * 2 ** 32 + 0.5) / 2 ** 32
    y = torch.where(_kept(s), x * (1.0 / (1.0 - p)), torch.zeros_like(x))
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(s["x"].dtype)}


def _bucket_of(s, delta):
    """Row of the bias for a query `delta` places behind its key."""
    b = s["case"]["buckets"]
    row = torch.searchsorted(s["starts"], delta.abs(), right=True) - 1
    if not s["case"].get("causal", True):
        row = torch.where(delta < 0, row + b, row)
    return row


def _plain_scores(s, q, k, h, t0, n):
    """Scores [m, n, n] of key head h of the history at t0, and the biases' rows of its pairs."""
    case = s["case"]
    m = case["hq"] // case["hk"]
    x = torch.matmul(q.reshape(m * n, -1), k.t().contiguous()).reshape(m, n, n) * s["scale"]
    at = torch.arange(n, device=x.device)
    delta = at[:, None] - at[None, :]
    rows = None
    if s["bias"] is not None:
        rows = _bucket_of(s, torch.arange(-(n - 1), n, device=x.device))[delta + n - 1]
        for i in range(m):
            x[i] += s["bias"][:, h * m + i][rows]
    if case["causal"]:
        x = x.masked_fill(delta < 0, float("-inf"))
    return x, rows


def _plain_attend(s):
    case = s["case"]
    hk, m = case["hk"], case["hq"] // case["hk"]
    out = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    t0 = 0
    for n in s["lens"]:
        for h in range(hk):
            q = s["q"][t0:t0 + n, h * m:(h + 1) * m].float().transpose(0, 1).contiguous()
            x, _ = _plain_scores(s, q, s["k"][t0:t0 + n, h].float(), h, t0, n)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.reshape(m * n, n), s["v"][t0:t0 + n, h].float()).reshape(m, n, -1) / total
            out[t0:t0 + n, h * m:(h + 1) * m] = o.transpose(0, 1)
            lse[t0:t0 + n, h * m:(h + 1) * m] = (top + torch.log(total))[..., 0].t()
        t0 += n
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_attend_back(s):
    case = s["case"]
    hk, m = case["hk"], case["hq"] // case["hk"]
    dt = s["q"].dtype
    res = {"dq": torch.empty(s["q"].shape, dtype=dt, device="cuda"),
           "dk": torch.empty(s["k"].shape, dtype=dt, device="cuda"),
           "dv": torch.empty(s["v"].shape, dtype=dt, device="cuda")}
    db = None if s["bias"] is None else torch.zeros(s["bias"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    for n in s["lens"]:
        for h in range(hk):
            q = s["q"][t0:t0 + n, h * m:(h + 1) * m].float().transpose(0, 1).contiguous()
            do = s["dout"][t0:t0 + n, h * m:(h + 1) * m].float().transpose(0, 1).reshape(m * n, -1)
            k, v = s["k"][t0:t0 + n, h].float(), s["v"][t0:t0 + n, h].float()
            x, rows = _plain_scores(s, q, k, h, t0, n)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            dp = torch.matmul(do, v.t().contiguous()).reshape(m, n, n)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            flat_p, flat_ds = p.reshape(m * n, n), ds.reshape(m * n, n)
            res["dv"][t0:t0 + n, h] = torch.matmul(flat_p.t().contiguous(), do).to(dt)
            res["dk"][t0:t0 + n, h] = (torch.matmul(flat_ds.t().contiguous(), q.reshape(m * n, -1)) * s["scale"]).to(dt)
            dq = (torch.matmul(flat_ds, k) * s["scale"]).reshape(m, n, -1)
            res["dq"][t0:t0 + n, h * m:(h + 1) * m] = dq.transpose(0, 1).to(dt)
            if db is not None:
                # sums along the pairs of one distance, then of each bucket
                for i in range(m):
                    wide = torch.zeros(n * (2 * n + 1), dtype=torch.float32, device="cuda")
                    wide[:2 * n * n].view(n, 2 * n)[:, :n] = ds[i]
                    # read as rows one longer, row i starts i places earlier: columns are distances, and those of
                    # keys behind the query end up at the end of the row above
                    by = wide.view(n, 2 * n + 1).sum(0, dtype=torch.float64)
                    lag = torch.arange(2 * n + 1, device="cuda")
                    delta = torch.where(lag < n, -lag, 2 * n + 1 - lag)
                    db[:, h * m + i].index_add_(0, _bucket_of(s, delta), by)
        t0 += n
    if db is not None:
        res["dbias"] = db.float()
    return res


def _plain_step(s):
    case = s["case"]
    hk, m, page = case["hk"], case["hq"] // case["hk"], case["page"]
    D = case["dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // page)].long()
        k = s["kc"][pages].reshape(-1, hk, D)[:n].float().permute(1, 2, 0).contiguous()   # [hk, D, n]
        v = s["vc"][pages].reshape(-1, hk, D)[:n].float().transpose(0, 1).contiguous()    # [hk, n, D]
        x = torch.matmul(s["q"][b].float().reshape(hk, m, D), k).reshape(hk * m, n) * s["scale"]
        if s["bias"] is not None:
            x = x + s["bias"][_bucket_of(s, torch.arange(n - 1, -1, -1, device="cuda"))].t()
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        out[b] = torch.matmul(p.reshape(hk, m, n), v).reshape(hk * m, D) / total
        lse[b] = (top + torch.log(total))[:, 0]
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---- the library's operators ----------------------------------------------------------

def _run_own(s):
    from dlrm_sparse_embedding_amd import emb as E
    op = s["case"]["op"]
    if op == "norm":
        E.emb_layer_norm(s["x"], s["y"], s["w"], s["b"], s["eps"])
        return {"y": s["y"]}
    if op == "norm_back":
        E.emb_layer_norm_backward(s["x"], s["dy"], s["dx"], s["w"], s["eps"], s["ws"], s["dw"], s["db"])
        res = {"dx": s["dx"], "dw": s["dw"]}
        if s["db"] is not None:
            res["db"] = s["db"]
        return res
    if op == "drop":
        E.emb_dropout(s["x"], s["y"], s["case"]["p"], s["key"], step=s["step"], residual=s["r"])
        return {"y": s["y"]}
    if op == "attend":
        E.emb_history_attention(s["h"].handle, s["q"], s["k"], s["v"], s["out"], s["offsets"], bias=s["bias"],
                                lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "step":
        E.emb_history_step(s["h"].handle, s["cache"].handle, s["q"], s["out"], s["lens_dev"], s["table"], s["ws"],
                           bias=s["bias"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    E.emb_history_attention_backward(s["h"].handle, s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"],
                                     s["dk"], s["dv"], s["offsets"], s["ws"], bias=s["bias"], dbias=s["dbias"])
    res = {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if s["dbias"] is not None:
        res["dbias"] = s["dbias"]
    return res


_PLAIN = {"norm": _plain_norm, "norm_back": _plain_norm_back, "drop": _plain_drop, "attend": _plain_attend,
          "attend_back": _plain_attend_back, "step": _plain_step}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits ---------------------------------------------------------

def _exact_norm(x, w, b, eps):
    mean = x.mean(-1, keepdim=True)
    var = (x * x).mean(-1, keepdim=True) - mean * mean
    y = (x - mean) / (var + eps).sqrt() * w
    return y if b is None else y + b


def _exact_draws(case, key, step):
    """The 32 random bits of each element, in host integers."""
    rows, dim = case["rows"], case["dim"]
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    parts = []
    for second in (0, 1):
        unit, row = np.meshgrid(np.arange(-(-dim // 8), dtype=np.uint64), np.arange(rows, dtype=np.uint64))
        a, b, c = unit, row, np.uint64(step) & low
        d = (np.uint64(step) >> shift & np.uint64(0x7FFFFFFF)) | np.uint64(second << 31)
        for i in range(10):
            x, y = np.uint64(0xD2511F53) * a, np.uint64(0xCD9E8D57) * c
            a = y >> shift ^ b ^ np.uint64(key % 2 ** 32 + i * 0x9E3779B9 & 0xFFFFFFFF)
            c = x >> shift ^ d ^ np.uint64((key >> 32) + i * 0xBB67AE85 & 0xFFFFFFFF)
            b, d = y & low, x & low
        words = np.stack(np.broadcast_arrays(a, b, c, d), -1).astype("<u4")
        parts.append(words.view("<u2").reshape(rows, -1)[:, :dim].astype(np.uint64))
    return parts[0] << np.uint64(16) | parts[1]


def _exact_rows(case, delta):
    """Row of the bias from the definition: the largest k whose bound the distance reaches."""
    b, exact_, far = _bias_shape(case)
    d = delta.abs()
    row = d.clamp(max=exact_)
    for k in range(1, b - exact_):
        bound = Fraction(far, exact_) ** k
        near = round(exact_ * float(bound) ** (1 / (b - exact_)))
        first = next(x for x in range(near - 2, near + 4) if Fraction(x, exact_) ** (b - exact_) >= bound)
        row = row + (d >= first)
    return row if case.get("causal", True) else row + b * (delta < 0)


def _exact_head(q, k, v, table, case, scale):
    """One query head over one history in 64 bits."""
    n = q.shape[0]
    at = torch.arange(n, device=q.device)
    delta = at[:, None] - at[None, :]
    s = q @ k.t() * scale
    if table is not None:
        # the table's rows by distance, once for all of a diagonal
        by = table[_exact_rows(case, torch.arange(1 - n, n, device=q.device))]
        s = s + by.unfold(0, n, 1).flip(1)
    if case["causal"]:
        s = s.masked_fill(delta < 0, float("-inf"))
    z = torch.logsumexp(s, -1)
    return torch.exp(s - z[:, None]) @ v, z


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        return {"y": _exact_norm(s["x"].double(), s["w"].double(), None if s["b"] is None else s["b"].double(), s["eps"])}
    if op == "norm_back":
        x = s["x"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        b = torch.zeros_like(w).requires_grad_()
        dx, dw, db = torch.autograd.grad(_exact_norm(x, w, b, s["eps"]), (x, w, b), s["dy"].double())
        return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
    if op == "drop":
        t = math.floor(case["p"] * 2 ** 32 + 0.5)
        kept = torch.from_numpy(_exact_draws(case, s["key"], int(s["step"])) >= np.uint64(t)).cuda()
        y = torch.where(kept, s["x"].double(), 0.0) / (1.0 - t / 2 ** 32)
        return {"y": y if s["r"] is None else y + s["r"].double()}
    hq, m = case["hq"], case["hq"] // case["hk"]
    if op == "step":
        out, lse = [], []
        for b, n in enumerate(s["lens"]):
            at = torch.arange(n, device="cuda")
            pg = s["table"][b].long()[at // case["page"]]
            for h in range(hq):
                k, v = s["kc"][pg, at % case["page"], h // m].double(), s["vc"][pg, at % case["page"], h // m].double()
                x = (k * s["q"][b, h].double()).sum(-1) * s["scale"]
                if s["bias"] is not None:
                    x = x + s["bias"][:, h].double()[_exact_rows(case, n - 1 - at)]
                z = torch.logsumexp(x, 0)
                out.append((torch.exp(x - z)[:, None] * v).sum(0))
                lse.append(z)
        return {"out": torch.stack(out).reshape(s["q"].shape), "lse": torch.stack(lse).reshape(s["q"].shape[:2])}
    back = op == "attend_back"
    names = ["q", "k", "v"] + (["bias"] if s["bias"] is not None else [])
    grads = {"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t0 = 0
    for n in s["lens"]:
        rows = slice(t0, t0 + n)
        for h in range(hq):
            x = [s["q"][rows, h], s["k"][rows, h // m], s["v"][rows, h // m]]
            x += [s["bias"][:, h]] if s["bias"] is not None else []
            x = [t.double().contiguous().requires_grad_(back) for t in x]
            o, z = _exact_head(*x[:3], x[3] if s["bias"] is not None else None, case, s["scale"])
            if back:
                g = torch.autograd.grad(o, x, s["dout"][rows, h].double())
                grads["dq"][rows, h] = g[0]
                grads["dk"][rows, h // m] += g[1]
                grads["dv"][rows, h // m] += g[2]
                if s["bias"] is not None:
                    grads["dbias"][:, h] += g[3]
            else:
                out[rows, h], lse[rows, h] = o, z
        t0 += n
    return grads if back else {"out": out, "lse": lse}
