"""Refusals of the sequence operators (CPU): every bad call is turned away with
its status code and a message before anything reaches the device. The C entry
points are called with made-up addresses that are never dereferenced."""
import math

import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E

FAKE = 0x100000
OK, INVAL, DTYPE, WS = E.EMB_OK, E.EMB_E_INVAL, E.EMB_E_DTYPE, E.EMB_E_WORKSPACE


def rotary_rc(**kw):
    f = dict(rot=64, layout=0, scaling=0, reserved=0, base=1e4, factor=1.0, original_len=0.0, turns_low=0.0,
             turns_high=0.0, magnitude=1.0)
    f.update(kw)
    out = E.ctypes.c_void_p()
    rc = E.lib().emb_create_rotary(E.emb_rotary_desc(*f.values()), out)
    if rc == OK:
        E.emb_destroy_rotary(out)
    else:
        assert out.value is None and E.lib().emb_last_error()
    return rc


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=63), dict(rot=258), dict(rot=-2), dict(layout=2), dict(layout=-1), dict(scaling=5),
    dict(scaling=-1), dict(reserved=1), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(magnitude=0.0),
    dict(magnitude=math.nan), dict(scaling=1, factor=0.0), dict(scaling=1, factor=math.inf), dict(scaling=2, rot=2, factor=2.0),
    dict(scaling=3, factor=2.0, original_len=0.0, turns_low=1.0, turns_high=2.0),
    dict(scaling=3, factor=2.0, original_len=10.0, turns_low=0.0, turns_high=2.0),
    dict(scaling=4, factor=2.0, original_len=10.0, turns_low=2.0, turns_high=2.0),
])
def test_rotary_descriptor_rejects(kw):
    assert rotary_rc(**kw) == INVAL


def test_rotary_descriptor_accepts():
    assert rotary_rc() == OK
    assert rotary_rc(rot=256, layout=1, scaling=3, factor=16.0, original_len=8192.0, turns_low=1.0, turns_high=32.0) == OK
    E.lib().emb_destroy_rotary(None)


@pytest.fixture
def rot():
    r = E.Rotary(64)
    yield r.handle
    r.close()


def apply_args(**kw):
    a = dict(pos=FAKE, itype=E.EMB_I64, tokens=4, dtype=E.EMB_BF16, dim=64, q=FAKE, qts=256, qhs=64, qo=FAKE + 4096,
             qots=256, qohs=64, hq=4, k=FAKE, kts=64, khs=64, ko=FAKE + 8192, kots=64, kohs=64, hk=1)
    a.update(kw)
    return list(a.values())


BAD_HEADS = [
    (dict(pos=None), INVAL), (dict(pos=FAKE + 4), INVAL), (dict(itype=2), DTYPE), (dict(tokens=-1), INVAL),
    (dict(tokens=1 << 31), INVAL), (dict(dtype=3), DTYPE), (dict(dim=62), INVAL), (dict(dim=1025), INVAL),
    (dict(hq=-1), INVAL), (dict(hk=70000), INVAL), (dict(q=None), INVAL), (dict(q=FAKE + 1), INVAL),
    (dict(qts=-1), INVAL), (dict(qo=None), INVAL), (dict(qohs=63), INVAL), (dict(qots=255), INVAL),
    (dict(qo=FAKE, qots=512), INVAL), (dict(k=None), INVAL), (dict(kots=0), INVAL),
]


@pytest.mark.parametrize("kw,code", BAD_HEADS)
def test_rotary_and_norm_reject(rot, kw, code):
    L = E.lib()
    assert L.emb_rotary_apply(rot, *apply_args(**kw), 0, None) == code
    assert L.emb_qk_norm_rotary(rot, *apply_args(**kw), FAKE, FAKE, 1e-6, None) == code
    assert L.emb_last_error()
    assert L.emb_rotary_apply(None, *apply_args(), 0, None) == INVAL


def test_rotary_nothing_to_do(rot):
    L = E.lib()
    assert L.emb_rotary_apply(rot, *apply_args(tokens=0, pos=None), 0, None) == OK
    assert L.emb_rotary_apply(rot, *apply_args(hq=0, hk=0, q=None, k=None, pos=None), 0, None) == OK


def test_norm_rejects_weights_and_eps(rot):
    L = E.lib()
    assert L.emb_qk_norm_rotary(rot, *apply_args(), FAKE + 4, FAKE, 1e-6, None) == INVAL
    assert L.emb_qk_norm_rotary(rot, *apply_args(), FAKE, FAKE + 8, 1e-6, None) == INVAL
    for eps in (-1.0, math.nan, math.inf):
        assert L.emb_qk_norm_rotary(rot, *apply_args(), FAKE, FAKE, eps, None) == INVAL


def back(rot, ws=FAKE, n=None, dwq=FAKE, eps=1e-6, **kw):
    a = dict(pos=FAKE, itype=E.EMB_I64, tokens=4, dtype=E.EMB_BF16, dim=64, q=FAKE, qts=256, qhs=64, dy=FAKE, dyts=256,
             dyhs=64, dq=FAKE + 4096, dqts=256, dqhs=64, hq=4, k=FAKE, kts=64, khs=64, dyk=FAKE, dykts=64, dykhs=64,
             dk=FAKE + 8192, dkts=64, dkhs=64, hk=1)
    a.update(kw)
    need = E.emb_qk_norm_rotary_workspace_bytes(4, 4, 1, 64)
    return E.lib().emb_qk_norm_rotary_backward(rot, *a.values(), FAKE, FAKE, eps, ws, need if n is None else need + n,
                                               dwq, FAKE, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), INVAL), (dict(ws=FAKE + 8), INVAL), (dict(n=-1), WS), (dict(dwq=FAKE + 2), INVAL),
    (dict(eps=-1.0), INVAL), (dict(dy=None), INVAL), (dict(dyk=None), INVAL), (dict(dq=None), INVAL),
    (dict(dqhs=32), INVAL), (dict(dq=FAKE, dqts=512), INVAL), (dict(pos=None), INVAL), (dict(dtype=9), DTYPE),
])
def test_norm_backward_rejects(rot, kw, code):
    assert back(rot, **kw) == code


def test_norm_backward_workspace_sizes():
    f = E.emb_qk_norm_rotary_workspace_bytes
    assert f(0, 4, 1, 64) == 0 and f(-1, 4, 1, 64) == 0 and f(4, 4, 1, 2000) == 0 and f(4, -1, 1, 64) == 0
    assert 0 < f(1, 1, 0, 64) <= f(100000, 1, 0, 64) <= 2048 * 2 * 64 * 4


KV = dict(k=FAKE, v=FAKE + (1 << 20), kps=4096, kss=64, khs=1024, vps=4096, vss=64, vhs=1024, pages=10, page=16, heads=4,
          dim=64, dtype=E.EMB_BF16, error=FAKE)


def make_kv(**kw):
    f = dict(KV)
    f.update(kw)
    out = E.ctypes.c_void_p()
    rc = E.lib().emb_create_kv(E.emb_kv_desc(*f.values()), out)
    return rc, out.value


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INVAL), (dict(v=None), INVAL), (dict(k=FAKE + 1), INVAL), (dict(dtype=5), DTYPE), (dict(pages=0), INVAL),
    (dict(pages=1 << 31), INVAL), (dict(page=0), INVAL), (dict(page=(1 << 20) + 1), INVAL), (dict(heads=0), INVAL),
    (dict(heads=65536), INVAL), (dict(dim=0), INVAL), (dict(dim=1025), INVAL), (dict(kss=-1), INVAL),
    (dict(error=FAKE + 2), INVAL),
])
def test_cache_descriptor_rejects(kw, code):
    rc, h = make_kv(**kw)
    assert rc == code and h is None and E.lib().emb_last_error()


@pytest.fixture
def kv():
    rc, h = make_kv()
    assert rc == OK
    yield h
    E.emb_destroy_kv(h)


def append(kv, rot, **kw):
    a = dict(tokens=4, dtype=E.EMB_BF16, heads=4, dim=64, k=FAKE, kts=256, khs=64, v=FAKE, vts=256, vhs=64, offsets=FAKE,
             seqs=2, lens=FAKE, table=FAKE, width=3, pos=None, itype=E.EMB_I64, norm=0, wk=None, eps=0.0)
    a.update(kw)
    return E.lib().emb_kv_append(kv, rot, *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVAL), (dict(dtype=E.EMB_F32), DTYPE), (dict(heads=3), INVAL), (dict(dim=128), INVAL),
    (dict(k=None), INVAL), (dict(v=FAKE + 1), INVAL), (dict(offsets=None), INVAL), (dict(offsets=FAKE + 2), INVAL),
    (dict(seqs=0), INVAL), (dict(seqs=-1), INVAL), (dict(lens=None), INVAL), (dict(table=None), INVAL),
    (dict(width=-1), INVAL), (dict(itype=4), DTYPE), (dict(pos=FAKE + 4), INVAL), (dict(norm=1, wk=FAKE + 4), INVAL),
    (dict(norm=1, eps=-1.0), INVAL), (dict(wk=FAKE), INVAL), (dict(khs=-64), INVAL),
])
def test_append_rejects(kv, rot, kw, code):
    assert append(kv, rot, **kw) == code
    assert E.lib().emb_last_error()


def test_append_more_rejects(kv, rot):
    assert append(None, rot) == INVAL
    assert append(kv, None, pos=FAKE) == INVAL       # positions without a rotation
    assert append(kv, rot, tokens=0, seqs=0, lens=None, table=None, k=None, v=None) == OK
    wide = E.Rotary(128)
    assert append(kv, wide.handle) == INVAL           # rot > dim
    wide.close()


def attend(kv, n=0, **kw):
    a = dict(tokens=4, dtype=E.EMB_BF16, dim=64, q=FAKE, qts=512, qhs=64, out=FAKE, ots=512, ohs=64, hq=8, scale=0.1,
             offsets=FAKE, seqs=2, lens=FAKE, table=FAKE, width=3, go=FAKE, groups=1, pl=FAKE, pt=FAKE, pwidth=5, ws=FAKE)
    a.update(kw)
    need = E.emb_prefix_attention_workspace_bytes(kv, 4, 8, 1, 5, 3) if kv else 0
    return E.lib().emb_prefix_attention(kv, *a.values(), need + n, kw.get("lse", FAKE), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVAL), (dict(tokens=1 << 24), INVAL), (dict(dtype=E.EMB_F16), DTYPE), (dict(dim=128), INVAL),
    (dict(q=None), INVAL), (dict(q=FAKE + 8), INVAL), (dict(qts=516), INVAL), (dict(qhs=68), INVAL), (dict(out=FAKE + 2), INVAL),
    (dict(ohs=32), INVAL), (dict(hq=6), INVAL), (dict(hq=0), INVAL), (dict(hq=260), INVAL), (dict(scale=math.nan), INVAL),
    (dict(offsets=None), INVAL), (dict(seqs=0), INVAL), (dict(lens=None), INVAL), (dict(table=None), INVAL),
    (dict(go=None), INVAL), (dict(pl=None), INVAL), (dict(pt=None), INVAL), (dict(groups=0), INVAL), (dict(groups=-1), INVAL),
    (dict(pwidth=1 << 27), INVAL), (dict(width=1 << 27), INVAL), (dict(ws=None), INVAL), (dict(ws=FAKE + 8), INVAL),
    (dict(n=-1), WS),
])
def test_attention_rejects(kv, kw, code):
    assert attend(kv, **kw) == code
    assert E.lib().emb_last_error()


def test_attention_rejects_caches():
    for kw, code in ((dict(dtype=E.EMB_F32), DTYPE), (dict(dim=80), INVAL), (dict(kss=68), INVAL), (dict(v=FAKE + 8), INVAL)):
        rc, h = make_kv(**kw)
        assert rc == OK
        assert E.emb_prefix_attention_workspace_bytes(h, 4, 8, 1, 5, 3) == 0
        assert attend(h, dtype=kw.get("dtype", E.EMB_BF16), dim=kw.get("dim", 64)) == code
        E.emb_destroy_kv(h)
    assert attend(None) == INVAL
    assert E.lib().emb_check_kv_error(None, None) == INVAL


def test_attention_workspace_sizes(kv):
    f = E.emb_prefix_attention_workspace_bytes
    assert f(kv, 0, 8, 1, 5, 3) == 0 and f(kv, 4, 7, 1, 5, 3) == 0
    one = f(kv, 4, 8, 0, 0, 3)
    assert one % 256 == 0 and one >= 4 * 8 * 65 * 4
    assert f(kv, 4, 8, 1, 5, 3) > one
    # at most 64 parts
    assert f(kv, 4, 8, 1, 1 << 20, 1 << 20) <= 64 * 4 * 8 * 65 * 4 + 1024


def test_binding_checks_tensors():
    r = E.Rotary(16)
    q = torch.zeros(3, 2, 16)
    pos = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="device"):
        E.emb_rotary_apply(r.handle, pos, q, q)
    with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
        E.emb_rotary_apply(r.handle, pos, q.double(), q.double())
    with pytest.raises(ValueError):
        E.KVCache(torch.zeros(2, 4, 1, 16), torch.zeros(2, 4, 1, 8))
    with pytest.raises(ValueError, match="device"):
        E.KVCache(torch.zeros(2, 4, 1, 16), torch.zeros(2, 4, 1, 16))
    with pytest.raises(E.EmbError):
        E.Rotary(15)
    r.close()
