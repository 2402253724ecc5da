"""The attention of histories and its step over its own queries (CPU): out that starts where q does has q's strides, or
a block would write rows that another has yet to read."""
import pytest

from dlrm_sparse_embedding_amd import emb as E
from tests.test_history_abi import ATT, FAKE, INVAL, STEP, WS, cache, handle, rc_of

APART = dict(k=FAKE + (1 << 20), v=FAKE + (2 << 20))


@pytest.mark.parametrize("kw", [
    dict(qts=768, ots=512), dict(qts=512, ots=768), dict(qts=1024, qhs=128, ots=1024, ohs=64), dict(qts=640, qhs=64, ots=1024, ohs=128)])
def test_attention_rejects_other_strides(kw):
    h = handle()
    assert rc_of("emb_history_attention", dict(ATT, h=h, **APART), kw) == INVAL
    assert b"other strides" in E.lib().emb_last_error()
    E.emb_destroy_history(h)


def test_step_rejects_other_strides():
    h, kv = handle(), cache()
    few = dict(STEP, h=h, kv=kv)
    for kw in (dict(qts=768, ots=512), dict(qts=1024, qhs=128, ots=1024)):
        assert rc_of("emb_history_step", few, kw) == INVAL
        assert b"other strides" in E.lib().emb_last_error()
    # the same strides get as far as the workspace; so do those over one sequence or one head
    assert rc_of("emb_history_step", few, dict(n=8)) == WS
    assert rc_of("emb_history_step", few, dict(n=8, seqs=1, qts=768)) == WS
    E.emb_destroy_history(h)
    E.emb_destroy_kv(kv)
    h, kv = handle(hq=1, hk=1), cache(heads=1)
    assert rc_of("emb_history_step", dict(STEP, h=h, kv=kv), dict(n=8, qhs=128)) == WS
    E.emb_destroy_history(h)
    E.emb_destroy_kv(kv)
