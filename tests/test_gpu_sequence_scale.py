"""GPU tests of the attention's scale at its lower end: 0 weighs every slot alike, and the smallest scales count
where the products of queries and keys are as large as the type allows. Tolerances as in test_gpu_sequence.py;
a subnormal scale is half of 2^-149 off, times products below 2^128: 2^-22, inside its 128 u."""
import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from tests.test_gpu_sequence import attention_case, check_attention, i32, run_attention

pytestmark = pytest.mark.gpu

# q heads, cache heads, prefix: own blocks, the prefix' blocks of 32 rows and of 128
KINDS = {"own": (2, 2, None), "narrow": (2, 2, 100), "wide": (8, 2, 100)}


def case(dt, kind, size, seed=31):
    hq, hk, prefix = KINDS[kind]
    counts, lens = [2, 1] * 10, [9, 40] * 10
    groups = ([20], [prefix]) if prefix else ([], [])
    q, kc, vc, off, lens, table, groups = attention_case(dt, 64, hq, hk, 16, counts, lens, *groups, seed=seed, big=size)
    kc.mul_(size)
    return q, kc, vc, off, lens, table, groups


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dt,size", [("bf16", 1.0), ("bf16", 2.0 ** 58), ("f16", 100.0)])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_a_scale_of_zero(dt, size, kind, scale):
    q, kc, vc, off, lens, table, groups = case(dt, kind, size)
    cache = E.KVCache(kc, vc)
    out, lse = run_attention(cache, q, scale, i32(off), i32(lens), table, groups)
    check_attention(out, lse, q, kc, vc, 0.0, off, lens, table, groups, dt)
    # what is not finite stays what 0 times it is: query 3 (token 0 of sequence 2), and whoever sees slot 2 of sequence 1
    base, base_l = out.clone(), lse.clone()
    q[3, 0, 5] = float("inf")
    pg, sl = int(table[1][2 // 16]), 2
    kc[pg, sl, 1] = float("-inf")
    out, lse = run_attention(cache, q, scale, i32(off), i32(lens), table, groups)
    m = q.shape[1] // 2
    nan = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    nan[3, 0] = True
    nan[2, m:] = True
    assert torch.equal(torch.isnan(lse), nan) and torch.equal(torch.isnan(out).all(-1), nan)
    assert torch.equal(out[~nan], base[~nan]) and torch.equal(lse[~nan], base_l[~nan])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -127, -3.0 * 2.0 ** -128, 2.0 ** -140, 2.0 ** -149])
def test_the_smallest_scales(kind, scale):
    # products of some 2^116 to 2^123
    q, kc, vc, off, lens, table, groups = case("bf16", kind, 2.0 ** 58)
    top = float((q.double().abs().max() * kc.double().abs().max() * 64))
    assert top < 2.0 ** 127 and np.isfinite(top)
    cache = E.KVCache(kc, vc)
    out, lse = run_attention(cache, q, scale, i32(off), i32(lens), table, groups)
    check_attention(out, lse, q, kc, vc, scale, off, lens, table, groups, "bf16")
