"""GPU tests of the range of the bias' entries: from the one that hides down, a distance is not seen, and up to it the
attention, its gradient and its step keep to their 64-bit definitions. Tolerances as in test_gpu_history.py: a score's
error, and with it a weight's, has a term of the bias' magnitude."""
import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_gpu_history import Call, Step, U, half, n64

pytestmark = pytest.mark.gpu

SPEC = (16, 8, 30)


@pytest.mark.parametrize("entry", [-2.0 ** 13, -1e4, -65504.0, -1e6, -1e9])
@pytest.mark.parametrize("dt,dim,causal", [("bf16", 64, True), ("f16", 64, False), ("bf16", 128, True),
                                           ("f16", 128, True)])
def test_entries_from_the_limit_down_hide(dt, dim, causal, entry):
    c = Call(dt, dim, 2, 1, [70, 3, 1], causal, SPEC, "plain")
    c.bias[0] = entry                   # a history's first item sees nothing if causal, that of the last one anyway
    c.bias[10:14, 0] = entry
    if not causal:
        c.bias[16:, 1] = entry
    c.forward()
    c.check_forward()
    empty = torch.isneginf(c.lse)
    assert empty[73].all() and (c.out[empty] == 0).all()
    c.backward()
    c.check_backward()
    assert (c.dq[empty] == 0).all() and (c.dbias[0] == 0).all()
    assert (c.dv[73] == 0).all() and (c.dk[73] == 0).all()
    hidden = [t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv, c.dbias)]
    c.bias[c.bias <= E.EMB_HIDDEN_BIAS] = float("-inf")
    c.forward(), c.backward()
    assert all(torch.equal(x, y) for x, y in zip(hidden, (c.out, c.lse, c.dq, c.dk, c.dv, c.dbias)))


@pytest.mark.parametrize("level", [-8180.0, -1000.0, 8180.0])
@pytest.mark.parametrize("dt,dim,causal", [("bf16", 64, True), ("f16", 64, False), ("bf16", 128, True),
                                           ("f16", 128, True)])
def test_entries_up_to_the_limit_are_weighed(dt, dim, causal, level):
    c = Call(dt, dim, 2, 1, [150, 3, 1], causal, SPEC, "plain")
    c.bias.clamp_(-4, 4).add_(level)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    # the only key that a query sees has all of its weight: dv is the sum over its query heads
    want = n64(c.dout[153]).sum(0)
    off = 6 * U * abs(level) + half(dt)
    assert (np.abs(n64(c.dv[153, 0]) - want) <= off * np.abs(n64(c.dout[153])).sum(0) + half(dt) * np.abs(want) * 1.01).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_the_step_hides_from_the_same_entry_down(dt):
    s = Step(dt, 64, 4, 2, [300, 1, 40], 16, SPEC)
    s.bias[0], s.bias[9:12, 1] = E.EMB_HIDDEN_BIAS, -1e5
    s.run()
    s.check()
    assert (s.out[1] == 0).all() and torch.isneginf(s.lse[1]).all()
    s.bias.clamp_(-4, 4).sub_(8180)
    s.run()
    s.check()
    assert s.lse.isfinite().all()
