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


def test_the_step_of_a_history_of_both_directions():
    """A new item sees earlier ones only: the rows of the other direction have no part in its step."""
    s = Step("bf16", 64, 4, 2, [300, 1, 40], 16, SPEC)
    s.run()
    want = [s.out.clone(), s.lse.clone()]
    both = E.HistoryAttention(4, 2, 64, "bf16", causal=False, buckets=SPEC[0], exact=SPEC[1], far=SPEC[2])
    s.bias = torch.cat([s.bias, torch.full_like(s.bias, float("nan"))])
    s.h, old = both, s.h
    s.run()
    assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1])
    old.close()


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn on one stream, with eager work on the same workspace between."""
    a, b = Call("bf16", 64, 4, 2, [300, 77], True, SPEC, seed=1), Call("f16", 128, 2, 1, [129], False, SPEC, seed=2)
    ws = max(a.ws, b.ws, key=lambda t: t.numel())
    want, graphs = [], []
    for c in (a, b):
        want.append([t.clone() for t in [*c.forward(), *c.backward()]])
        c.ws = ws
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.forward(), c.backward()
    for i in (0, 1, 1, 0, 0, 1):
        c = (a, b)[i]
        got = [c.out, c.lse, c.dq, c.dk, c.dv, c.dbias]
        for t in got:
            t.fill_(3)
        graphs[i].replay()
        assert all(torch.equal(x, y) for x, y in zip(got, want[i]))
        (b, a)[i].backward()
        torch.cuda.synchronize()
