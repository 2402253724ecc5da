"""GPU tests of paths of the attention of histories and its gradient that short or narrow cases do not take: whole
64-query halves of the gradient's tiles (bf16 heads of 96 and 128) with biases of each distance and of both directions'
last buckets, several key tiles in both directions, the correction of the rows' sums, and the largest strides.
Tolerances as in test_gpu_history.py, but for the correction's test, which derives its own."""
import numpy as np
import pytest
import torch

from oracle import history_oracle as H
from tests.test_gpu_history import Call, U, close, half, n64

pytestmark = pytest.mark.gpu

LAST = (12, 4, 60)      # the last bucket starts inside these histories


def pairs(lens, causal, spec):
    """How many times (64 queries of a half tile that all see 32 keys) have the biases of each distance, the last bucket's
    of keys before them, and the last bucket's of keys behind them."""
    near = far = beyond = 0
    last = next(d for d in range(1 << 20) if H.bucket(d, *spec) == spec[0] - 1) if spec else 0
    for n in lens:
        for k0 in range(0, n, 32):
            begin = k0 // 128 * 128 if causal else 0
            for q in range(begin, n, 64):
                if q + 64 > n or (q < k0 + 31 if causal else k0 + 32 > n):
                    continue
                if not spec or q - 31 - k0 >= last:
                    far += 1
                elif not causal and q + 63 - k0 <= -last:
                    beyond += 1
                else:
                    near += 1
    return near, far, beyond


@pytest.mark.parametrize("dt,dim,hq,hk,lens,causal,spec", [
    ("bf16", 96, 4, 2, [300, 70], True, LAST),
    ("bf16", 96, 2, 1, [260], False, LAST),
    ("bf16", 96, 2, 2, [300, 131], True, None),
    ("bf16", 96, 2, 1, [300], False, None),
    ("bf16", 128, 2, 1, [500], False, LAST),
    ("bf16", 128, 4, 2, [300, 200], False, None),
    ("bf16", 128, 4, 1, [450, 64, 90], True, LAST),
    ("f16", 128, 2, 1, [300], False, LAST),
    ("f16", 96, 4, 2, [300, 70], True, LAST),
    ("f16", 128, 2, 2, [300, 131], False, None),
    ("bf16", 64, 4, 2, [300, 131], False, LAST),
])
def test_whole_halves_of_tiles(dt, dim, hq, hk, lens, causal, spec):
    near, far, beyond = pairs(lens, causal, spec)
    assert far and (not spec or near and (causal or beyond))
    c = Call(dt, dim, hq, hk, lens, causal, spec, "wide")
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
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
    c.h.check_error()


@pytest.mark.parametrize("dt,dim,causal,spec", [
    ("bf16", 64, True, None), ("bf16", 64, False, LAST), ("bf16", 96, True, LAST), ("bf16", 128, True, LAST),
    ("bf16", 128, False, None)])
def test_gradient_of_queries_is_corrected_for_the_rounding_of_out(dt, dim, causal, spec):
    """Values and keys with a large part in common: rounding `out` to its type moves dout . out, with which a row's sum
    of P dP starts, by about as much as dS itself, and a dq made from that sum by `mistake` = scale (dout . (out - its
    exact value)) sum P k. After the correction there remain, with h half a step of the type, slip the size of that
    shift, and per row over its keys:
      - dS, shift included, rounded for the product: h (sum |dS| |k| + slip sum P |k|);
      - P rounded in the product that is taken off: h slip sum P |k|;
      - P off by 2 e relative through the scores: 2 e (sum |dS| |k| + sum |dS| sum P |k|);
      - dP and the sums in fp32: (D + 600) u sum P (|dP| + sum P |dP|) |k|, |.| magnitudes; and h of the result."""
    n = 200
    c = Call(dt, dim, 2, 1, [n], causal, spec, "plain")
    gen = torch.Generator().manual_seed(dim)
    for t, by in ((c.v, 16.0), (c.k, 3.0)):
        t.copy_(t.float() + by * (1 + torch.rand((1, 1, dim), generator=gen)).cuda())
    c.forward()
    c.backward()
    q, k, v = c.arrays()
    do, out, bias = n64(c.dout), n64(c.out), n64(c.bias)
    want = np.zeros_like(do)
    tol, mistake = np.zeros_like(do), np.zeros_like(do)
    h, e = half(dt), c.score_error()
    for i in range(2):
        s, _ = H.scores(q[:, i], k[:, 0], c.scale, causal, None if bias is None else bias[:, i], spec)
        p, _ = H.softmax(s)
        dp, adp = do[:, i] @ v[:, 0].T, np.abs(do[:, i]) @ np.abs(v[:, 0]).T
        ds = p * (dp - (p * dp).sum(1, keepdims=True))
        mag = p * (adp + (p * adp).sum(1, keepdims=True))
        ak = np.abs(k[:, 0])
        off = (do[:, i] * (out[:, i] - p @ v[:, 0])).sum(1, keepdims=True)
        slip, pk = np.abs(off), p @ ak
        want[:, i] = c.scale * (ds @ k[:, 0])
        mistake[:, i] = c.scale * np.abs(off * (p @ k[:, 0]))
        tol[:, i] = c.scale * (h * (np.abs(ds) @ ak + 2 * slip * pk) +
                               2 * e * (np.abs(ds) @ ak + np.abs(ds).sum(1, keepdims=True) * pk) +
                               (dim + 600) * U * (mag @ ak))
    tol += h * np.abs(want)
    assert (mistake > 2 * tol).mean() > 0.05         # a dq without the correction would show
    close(c.dq, want, tol, dt, "dq")


def test_the_largest_strides():
    """Tokens 2^24 - 8 elements apart, the most that a call takes: the rows of a tile span nearly 2^32 bytes."""
    n, ts = 170, (1 << 24) - 8
    for dim, spec in ((64, (32, 16, 128)), (128, None)):
        c = Call("bf16", dim, 1, 1, [n], True, spec, "plain")
        c.forward(), c.backward()
        want = [t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv)]
        dbias = None if spec is None else c.dbias.clone()
        base = torch.empty(n * ts, dtype=torch.bfloat16, device="cuda")
        far = [base.as_strided((n, 1, dim), (ts, dim, 1), dim * i) for i in range(8)]
        for x, t in zip(far, (c.q, c.k, c.v, c.dout)):
            x.copy_(t)
        c.q, c.k, c.v, c.dout, c.out, c.dq, c.dk, c.dv = far
        c.forward(), c.backward()
        assert all(torch.equal(x, y) for x, y in zip(want, (c.out, c.lse, c.dq, c.dk, c.dv)))
        assert dbias is None or torch.equal(dbias, c.dbias)
