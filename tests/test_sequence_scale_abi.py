"""Refusals of the attention's scale (CPU): its product with log2(e) has to fit fp32. The entry point is called
without tokens, so nothing reaches the device."""
import math

import pytest

from dlrm_sparse_embedding_amd import emb as E
from tests.test_sequence_abi import FAKE, make_kv


@pytest.mark.parametrize("scale,code", [
    (0.0, E.EMB_OK), (-0.0, E.EMB_OK), (2.0 ** -149, E.EMB_OK), (2.0 ** 127, E.EMB_OK), (-2.0 ** 127, E.EMB_OK),
    (2.0 ** 127 * 1.01, E.EMB_E_INVAL), (-3.0e38, E.EMB_E_INVAL), (math.inf, E.EMB_E_INVAL), (math.nan, E.EMB_E_INVAL),
])
def test_scales(scale, code):
    rc, kv = make_kv()
    assert rc == E.EMB_OK
    got = E.lib().emb_prefix_attention(kv, 0, E.EMB_BF16, 64, FAKE, 512, 64, FAKE, 512, 64, 8, scale, FAKE, 2, FAKE, FAKE, 3,
                                       None, 0, None, None, 0, FAKE, 0, None, None)
    E.emb_destroy_kv(kv)
    assert got == code
