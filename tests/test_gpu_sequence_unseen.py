"""GPU test that slots which a query does not see change no bit of its result, before the rounding to 16 bits
too: the partial outputs of a call are fp32 and stay in its workspace."""
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_gpu_sequence import attention_case, i32

pytestmark = pytest.mark.gpu


def parts_of(nbytes, rows, D):
    """How many partial outputs a workspace of this size has for each of its rows (fp32, with a log-sum each)."""
    up = lambda n: -(-n // 256) * 256
    parts = nbytes // (rows * (D + 1) * 4)
    assert nbytes == up(rows * parts * D * 4) + up(rows * parts * 4)
    return parts


# q heads, cache heads, length of the prefix: 24 queries of one sequence in own blocks (their table is wide), in
# the prefix' blocks of 32 rows, in those of 128
KINDS = {"own": (2, 2, None), "narrow": (2, 2, 1500), "wide": (8, 2, 1500)}


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 96)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_unseen_values_change_no_bit(dt, D, kind):
    hq, hk, prefix = KINDS[kind]
    n, lens = 24, 60
    q, kc, vc, off, _, table, groups = attention_case(dt, D, hq, hk, 16, [n], [lens], [1] if prefix else [],
                                                      [prefix] if prefix else [])
    table = table[:, :4].contiguous()                # 64 slots of table width
    if not prefix:
        table = torch.cat([table, torch.full((1, 60), -1, dtype=torch.int32, device="cuda")], 1)
    cache = E.KVCache(kc, vc)
    go, pl, pt = groups if prefix else (None, None, None)
    size = E.emb_prefix_attention_workspace_bytes(cache.handle, n, hq, 1 if prefix else 0, pt.shape[1] if prefix else 0,
                                                  table.shape[1])
    parts = parts_of(size, n * hq, D)
    assert parts > 2, "the result would not go through partial outputs"

    def run():
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((n, hq), device="cuda")
        E.emb_prefix_attention(cache.handle, q, out, 0.125, i32(off), i32([lens]), table, go, pl, pt, ws, lse=lse)
        cache.check_error()
        return ws[:parts * n * hq * D * 4].view(torch.int32).reshape(parts, n, hq, D), out, lse

    o0, out0, lse0 = run()
    for s in (lens - 1, lens - 2, lens - 9):          # seen by the last, the last two, the last nine queries
        seen = lens - s
        pg, sl = int(table[0][s // 16]), s % 16
        keep = kc[pg, sl].clone(), vc[pg, sl].clone()
        for poison in (float("inf"), float("-inf"), float("nan")):
            vc[pg, sl] = poison
            o, out, lse = run()
            assert torch.equal(o[:, :n - seen], o0[:, :n - seen]), (s, poison)
            assert torch.equal(out[:n - seen], out0[:n - seen]) and torch.equal(lse, lse0)
            assert not torch.isfinite(out[n - seen:]).any()
            kc[pg, sl] = poison
            o, out, lse = run()
            assert torch.equal(o[:, :n - seen], o0[:, :n - seen]) and torch.equal(lse[:n - seen], lse0[:n - seen])
            kc[pg, sl], vc[pg, sl] = keep
