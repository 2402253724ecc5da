"""GPU tests of what calls on a paged cache report: offsets that break their contract inside as well as at
their ends, and lengths that a page table does not hold. Every input here stays inside the buffers, and no two
tokens of an append meet in a slot."""
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


# ---- the attention -------------------------------------------------------------------------
# 8 tokens: with 2 query heads of a cache head 16 rows, in tiles of 32 (narrow), with 32 of them 256 rows, in
# tiles of 128 that share their keys (wide)

KERNELS = {"narrow": (4, 2), "wide": (64, 2)}


def attention(hq, hk, off, groups=None, counts=(3, 2, 3), lens=(9, 40, 5), prefix=(70,)):
    q, kc, vc, _, _, table, good = attention_case("bf16", 64, hq, hk, 16, list(counts), list(lens), [len(lens)], list(prefix))
    cache = E.KVCache(kc, vc)
    run_attention(cache, q, 0.125, i32(off), i32(lens), table, groups(good) if groups else None)
    return reported(cache)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("own_blocks", [False, True])
@pytest.mark.parametrize("off,code", [
    ([0, 3, 5, 8], 0),
    ([0, 5, 3, 8], E.EMB_E_INVAL),             # decreasing inside
    ([0, 3, 2147483647, 8], E.EMB_E_INVAL),
    ([0, -1, 5, 8], E.EMB_E_INVAL),
    ([0, 3, 5, 9], E.EMB_E_INVAL),
    ([1, 3, 5, 8], E.EMB_E_INVAL),
])
def test_attention_reports_offsets(kernel, own_blocks, off, code):
    hq, hk = KERNELS[kernel]
    assert attention(hq, hk, off, groups=None if own_blocks else lambda good: good) == code


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_attention_reports_offsets_of_groups(kernel):
    hq, hk = KERNELS[kernel]
    _, pl, pt = attention_case("bf16", 64, hq, hk, 16, [3, 2, 3], [9, 40, 5], [3], [70])[6]
    run = lambda go: attention(hq, hk, [0, 3, 5, 8], groups=lambda good: (
        i32(go), pl.repeat(len(go) - 1), pt.repeat(len(go) - 1, 1)))
    assert run([0, 1, 1, 3]) == 0
    # decreasing inside; beyond the sequences, where they are cut, so no two groups share a row
    assert run([0, 5, 3]) == E.EMB_E_INVAL
    assert run([0, 5, 4, 3]) == E.EMB_E_INVAL
    assert run([0, -1, 3]) == E.EMB_E_INVAL


def test_attention_reports_offsets_of_many_groups():
    # more groups than a wave has lanes, and than a block has threads
    hq, hk = 4, 2
    counts, lens = [1] * 400, [3] * 400
    q, kc, vc, _, _, table, _ = attention_case("bf16", 64, hq, hk, 16, counts, lens, [400], [40])
    cache = E.KVCache(kc, vc)
    pages = torch.arange(3, dtype=torch.int32, device="cuda")[None].repeat(400, 1)
    good = list(range(401))
    beyond = good[:300] + [400] * 101
    beyond[350] = 450                     # cut to the sequences: no group shares a row
    last = good[:399] + [407, 400]
    for go, code in ((good, 0), (beyond, E.EMB_E_INVAL), (last, E.EMB_E_INVAL)):
        run_attention(cache, q, 0.125, None, i32(lens), table, (i32(go), i32([40] * 400), pages))
        assert reported(cache) == code


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_attention_reports_prefixes_that_their_tables_do_not_hold(kernel):
    hq, hk = KERNELS[kernel]
    off = [0, 3, 5, 8]
    table_of = lambda n: torch.zeros((1, n), dtype=torch.int32, device="cuda")
    run = lambda n, width, go=(0, 3): attention(hq, hk, off, groups=lambda good: (
        i32(go), i32(n), table_of(width).repeat(len(n), 1)))
    assert run([32], 2) == 0 and run([0], 0) == 0 and run([0], 2) == 0
    assert run([33], 2) == E.EMB_E_BOUNDS
    assert run([-1], 2) == E.EMB_E_BOUNDS
    assert run([5], 0) == E.EMB_E_BOUNDS          # no page at all: nothing but the lengths tells
    assert run([-1], 0) == E.EMB_E_BOUNDS
    assert run([0, 9], 0, (0, 3, 3)) == E.EMB_E_BOUNDS
    # the same of a group without sequences, among few and among many
    assert run([16, 99], 2, (0, 3, 3)) == E.EMB_E_BOUNDS
    assert run([16] + [0] * 300, 2, [0] + [3] * 301) == 0
    assert run([16] + [0] * 299 + [99], 2, [0] + [3] * 301) == E.EMB_E_BOUNDS
