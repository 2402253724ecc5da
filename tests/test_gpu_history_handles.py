"""GPU test of the attention of histories through a handle of emb_create_history."""
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_gpu_history import SPEC, Call, Step

pytestmark = pytest.mark.gpu


def test_a_created_handle_gives_the_same_bits():
    c = Call("f16", 64, 4, 2, [70, 3], False, SPEC)
    want = [t.clone() for t in [*c.forward(), *c.backward()]]
    s = Step("f16", 64, 4, 2, [70, 3], 16, SPEC)
    s.run()
    step = s.out.clone()
    for t in (c.out, c.lse, c.dq, c.dk, c.dv, s.out):
        t.fill_(3)
    mine = [E.emb_create_history(E.emb_history_desc(4, 2, 64, E.EMB_F16, causal, *SPEC, 64 ** -0.5, 0, None))
            for causal in (0, 1)]
    with pytest.raises(ValueError):
        E.emb_history_attention(mine[1], c.q, c.k, c.v, c.out, c.offsets, bias=c.bias)     # twice the rows of its bias
    E.emb_history_attention(mine[0], c.q, c.k, c.v, c.out, c.offsets, bias=c.bias, lse=c.lse)
    E.emb_history_attention_backward(mine[0], c.q, c.k, c.v, c.out, c.lse, c.dout, c.dq, c.dk, c.dv, c.offsets, c.ws,
                                     bias=c.bias, dbias=c.dbias)
    assert all(torch.equal(x, y) for x, y in zip(want, (c.out, c.lse, c.dq, c.dk, c.dv, c.dbias)))
    E.emb_history_step(mine[1], s.cache.handle, s.q, s.out, s.lens, s.table, s.ws, bias=s.bias)
    assert torch.equal(s.out, step)
    E.emb_check_history_error(mine[0])
    for h in mine:
        E.emb_destroy_history(h)
