"""GPU tests of what calls on a paged cache report: offsets that break their contract inside as well as at
their ends, and lengths that a page table does not hold. Every input here stays inside the buffers, and no two
tokens of an append meet in a slot."""
import math

import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_gpu_sequence import attention_case, i32, paged, randn, run_attention

pytestmark = pytest.mark.gpu


def reported(cache):
    """The code of the report, 0 where there is none; the report is gone afterwards."""
    try:
        cache.check_error()
    except E.EmbError as e:
        cache.check_error()
        return e.code
    return 0


# ---- the append ------------------------------------------------------------------------

@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 72)])       # 16-byte units, element by element
@pytest.mark.parametrize("off", [
    [0, 5, 3, 8],      # decreasing inside
    [0, 3, 5, 9],      # more tokens than there are
    [-2, 3, 5, 8],     # from before the first
    [0, 3, 5, 7],      # the last token in no sequence
    [1, 3, 5, 8],      # the first in none
    [0, 3, 2147483647, 8],
])
def test_append_reports_offsets(dt, D, off):
    gen = torch.Generator().manual_seed(71)
    kc, vc = paged(gen, dt, 8, 16, 2, D)
    k, v = randn(gen, (8, 2, D), dt), randn(gen, (8, 2, D), dt)
    table, lens = torch.tensor([[6], [1], [4]], dtype=torch.int32).cuda(), i32([10, 10, 10])
    cache = E.KVCache(kc, vc)
    k0 = kc.clone()
    E.emb_kv_append(cache.handle, None, k, v, i32(off), lens, table)
    assert reported(cache) == E.EMB_E_INVAL
    other = [0, 2, 3, 5, 7]
    assert torch.equal(kc[other], k0[other]), "pages of no sequence"
    if off[:2] == [0, 3]:      # sequence 0's own offsets are in order
        assert torch.equal(kc[6, 7:10], k[:3])
    if off[3] == 9 or off[0] == -2:      # a sequence with tokens that are not there: nothing is stored at shifted slots
        page = 4 if off[3] == 9 else 6
        assert torch.equal(kc[page], k0[page])


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 72)])
def test_append_reports_no_good_offsets(dt, D):
    gen = torch.Generator().manual_seed(72)
    n = 700                    # more sequences than one block has threads, most without tokens
    kc, vc = paged(gen, dt, 4, 16, 2, D)
    k, v = randn(gen, (2, 2, D), dt), randn(gen, (2, 2, D), dt)
    table = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    table[3], table[650] = 2, 1
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    lens[3], lens[650] = 5, 9
    off = [0] * 4 + [1] * 647 + [2] * 50
    assert len(off) == n + 1
    cache = E.KVCache(kc, vc)
    E.emb_kv_append(cache.handle, None, k, v, i32(off), lens, table)
    assert reported(cache) == 0
    assert torch.equal(kc[2, 4], k[0]) and torch.equal(kc[1, 8], k[1])
    off[680] = 1               # far behind the last token
    E.emb_kv_append(cache.handle, None, k, v, i32(off), lens, table)
    assert reported(cache) == E.EMB_E_INVAL
