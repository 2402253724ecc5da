"""GPU tests of paths of the attention of histories and its gradient that short or narrow cases do not take: whole
64-query halves of the gradient's tiles (bf16 heads of 96 and 128) with biases of each distance and of both directions'
last buckets, and several key tiles in both directions. Tolerances as in test_gpu_history.py."""
import pytest
import torch

from oracle import history_oracle as H
from tests.test_gpu_history import Call

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
