"""GPU tests of queries that see no key because the bias hides all of them."""
import pytest
import torch

from tests.test_gpu_history import SPEC, Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,dim,causal", [("bf16", 64, True), ("f16", 96, True), ("bf16", 128, True), ("f16", 128, False)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_sees_nothing_gets_zeros_whatever_values_hold(dt, dim, causal, bad):
    """One head sees nothing, the other all: values that are no numbers reach the rows of the second alone."""
    c = Call(dt, dim, 2, 1, [150, 9], causal, SPEC, "plain")
    c.bias[:, 0] = float("-inf")
    at = 77
    c.v[at, 0, 5] = bad
    c.forward()
    assert (c.out[:, 0] == 0).all() and torch.isneginf(c.lse[:, 0]).all()
    seen = c.out[at if causal else 0:150, 1, 5]
    assert not seen.isfinite().any() and c.out[150:].isfinite().all() and c.lse[:, 1].isfinite().all()
    rest = c.out[:, 1].clone()
    rest[at if causal else 0:150, 5] = 0
    assert rest.isfinite().all()
