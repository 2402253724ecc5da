"""GPU tests of the attention of histories and its step written over their own queries: the bits of the call apart."""
import pytest
import torch

from tests.test_gpu_history import SPEC, Call, Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,dim,causal,memory", [("bf16", 128, True, "fused"), ("f16", 64, False, "wide"),
                                                  ("bf16", 96, True, "heads_first")])
def test_attention_over_its_queries(dt, dim, causal, memory):
    c = Call(dt, dim, 4, 2, [300, 0, 1, 129], causal, SPEC, memory)
    c.forward()
    want = [c.out.clone(), c.lse.clone()]
    c.out = c.q
    c.forward()
    assert torch.equal(c.q, want[0]) and torch.equal(c.lse, want[1])


@pytest.mark.parametrize("lens", [[700, 90], [20] * 600])       # parts that are joined, and one part each
def test_step_over_its_queries(lens):
    s = Step("bf16", 64, 4, 2, lens, 16, SPEC)
    s.run()
    want = s.out.clone()
    s.out = s.q
    s.run()
    assert torch.equal(s.q, want)
