"""Refusals of the history layer (CPU): every bad call is turned away with its status code and a message before
anything reaches the device. The C entry points are called with made-up addresses that are never dereferenced."""
import math

import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E

FAKE = 0x100000
OK, INVAL, DTYPE, WS = E.EMB_OK, E.EMB_E_INVAL, E.EMB_E_DTYPE, E.EMB_E_WORKSPACE


def rc_of(name, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    rc = getattr(E.lib(), name)(*a.values())
    assert rc == OK or E.lib().emb_last_error()
    return rc


NORM = dict(rows=4, dim=64, x=FAKE, xt=E.EMB_BF16, xs=64, y=FAKE + 4096, yt=E.EMB_BF16, ys=64, w=FAKE, b=FAKE, eps=1e-5,
            st=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVAL), (dict(rows=1 << 31), INVAL), (dict(dim=0), INVAL), (dict(dim=-3), INVAL),
    (dict(dim=16385), INVAL), (dict(xt=3), DTYPE), (dict(yt=-1), DTYPE), (dict(yt=E.EMB_F32), DTYPE),
    (dict(yt=E.EMB_F16), DTYPE), (dict(x=None), INVAL), (dict(y=None), INVAL), (dict(x=FAKE + 1), INVAL),
    (dict(xt=E.EMB_F32, x=FAKE + 2), INVAL), (dict(y=FAKE + 1), INVAL), (dict(xs=-64), INVAL), (dict(ys=63), INVAL),
    (dict(ys=0), INVAL), (dict(w=FAKE + 4), INVAL), (dict(b=FAKE + 8), INVAL), (dict(eps=-1.0), INVAL),
    (dict(eps=math.nan), INVAL), (dict(eps=math.inf), INVAL), (dict(y=FAKE, xs=128), INVAL),
    (dict(xt=E.EMB_F32, y=FAKE), INVAL),
])
def test_layer_norm_rejects(kw, code):
    assert rc_of("emb_layer_norm", NORM, kw) == code


def test_layer_norm_without_rows_is_ok():
    assert rc_of("emb_layer_norm", NORM, dict(rows=0, x=None, y=None, w=None, b=None)) == OK


BACK = dict(rows=4, dim=64, x=FAKE, xt=E.EMB_F32, xs=64, dy=FAKE + 4096, yt=E.EMB_BF16, dys=64, dx=FAKE + 8192, dxs=64,
            w=FAKE, eps=1e-5, ws=FAKE, n=1 << 20, dw=FAKE, db=FAKE, st=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVAL), (dict(dim=16385), INVAL), (dict(xt=E.EMB_BF16, yt=E.EMB_F32), DTYPE), (dict(x=None), INVAL),
    (dict(dy=None), INVAL), (dict(dx=None), INVAL), (dict(dxs=8), INVAL), (dict(dx=FAKE + 2), INVAL),
    (dict(dys=-1), INVAL), (dict(ws=None), INVAL), (dict(ws=FAKE + 8), INVAL), (dict(n=4 * 2 * 64 * 4 - 1), WS),
    (dict(dw=FAKE + 2), INVAL), (dict(db=FAKE + 1), INVAL), (dict(dx=FAKE + 4096), INVAL), (dict(dx=FAKE, xs=128), INVAL),
    (dict(w=FAKE + 4), INVAL), (dict(eps=-0.5), INVAL),
])
def test_layer_norm_backward_rejects(kw, code):
    assert rc_of("emb_layer_norm_backward", BACK, kw) == code


def test_layer_norm_workspace():
    f = E.emb_layer_norm_workspace_bytes
    assert f(4, 64) == 4 * 2 * 64 * 4 and f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 16385) == 0
    for dim in (1, 64, 1000, 1025, 4096, 16384):
        assert f((1 << 31) - 1, dim) <= 64 << 20


DROP = dict(rows=4, dim=64, t=E.EMB_BF16, x=FAKE, xs=64, r=FAKE + 4096, rs=64, y=FAKE + 8192, ys=64, p=0.1, seed=1,
            step=FAKE, st=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVAL), (dict(rows=1 << 31), INVAL), (dict(dim=0), INVAL), (dict(t=5), DTYPE), (dict(x=None), INVAL),
    (dict(y=None), INVAL), (dict(x=FAKE + 1), INVAL), (dict(r=FAKE + 1), INVAL), (dict(xs=-1), INVAL),
    (dict(rs=-1), INVAL), (dict(ys=32), INVAL), (dict(p=-0.1), INVAL), (dict(p=1.1), INVAL), (dict(p=math.nan), INVAL),
    (dict(step=FAKE + 4), INVAL), (dict(y=FAKE, xs=128), INVAL), (dict(y=FAKE + 4096, rs=0), INVAL),
])
def test_dropout_rejects(kw, code):
    assert rc_of("emb_dropout", DROP, kw) == code


def test_dropout_without_rows_is_ok():
    assert rc_of("emb_dropout", DROP, dict(rows=0, x=None, y=None)) == OK


def test_binding_checks_shapes_and_types():
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError):
        E.emb_layer_norm(torch.zeros(8), x, None, None, 0.0)
    with pytest.raises(ValueError):
        E.emb_layer_norm(x, x, None, None, 0.0)               # not in device memory
    with pytest.raises(ValueError):
        E.emb_dropout(x.double(), x, 0.1, 0)


# ---- attention of histories ---------------------------------------------------------

DESC = dict(hq=8, hk=2, dim=64, t=E.EMB_BF16, causal=1, buckets=32, exact=16, far=128, scale=0.125, reserved=0, error=None)


def history_rc(**kw):
    f = dict(DESC)
    f.update(kw)
    out = E.ctypes.c_void_p()
    rc = E.lib().emb_create_history(E.emb_history_desc(*f.values()), out)
    if rc == OK:
        E.emb_destroy_history(out)
    else:
        assert out.value is None and E.lib().emb_last_error()
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(t=E.EMB_F32), DTYPE), (dict(t=9), DTYPE), (dict(dim=32), INVAL), (dict(dim=256), INVAL), (dict(hk=0), INVAL),
    (dict(hq=0), INVAL), (dict(hq=7), INVAL), (dict(hq=130), INVAL), (dict(hq=65536, hk=65536), INVAL),
    (dict(scale=0.0), INVAL), (dict(scale=-1.0), INVAL), (dict(scale=math.nan), INVAL), (dict(scale=math.inf), INVAL),
    (dict(buckets=-1), INVAL), (dict(buckets=129), INVAL), (dict(exact=0), INVAL), (dict(exact=33), INVAL),
    (dict(far=16), INVAL), (dict(far=(1 << 30) + 1), INVAL), (dict(buckets=0), INVAL), (dict(reserved=1), INVAL),
    (dict(error=FAKE + 2), INVAL),
])
def test_history_descriptor_rejects(kw, code):
    assert history_rc(**kw) == code


def test_history_descriptor_accepts():
    assert history_rc() == OK
    assert history_rc(buckets=0, exact=0, far=0) == OK
    assert history_rc(buckets=128, exact=128, far=0, causal=0) == OK
    assert history_rc(buckets=128, exact=1, far=1 << 30) == OK
    E.lib().emb_destroy_history(None)
    assert E.lib().emb_create_history(None, None) == INVAL


def handle(**kw):
    f = dict(DESC)
    f.update(kw)
    return E.emb_create_history(E.emb_history_desc(*f.values()))


def cache(dim=64, heads=2, dtype=E.EMB_BF16, k=FAKE, slot=64):
    return E.emb_create_kv(E.emb_kv_desc(k, FAKE, 16 * heads * dim, slot, 16 * dim, 16 * heads * dim, slot, 16 * dim,
                                         100, 16, heads, dim, dtype, None))


ATT = dict(h=None, tokens=10, q=FAKE, qts=768, qhs=64, k=FAKE, kts=768, khs=64, v=FAKE, vts=768, vhs=64, out=FAKE,
           ots=512, ohs=64, off=FAKE, seqs=2, bias=FAKE, lse=FAKE, st=None)
BAD_RAGGED = [
    dict(h=0), dict(tokens=-1), dict(tokens=1 << 24), dict(seqs=-1), dict(seqs=0), dict(seqs=1 << 24), dict(bias=None),
    dict(bias=FAKE + 2), dict(off=None), dict(off=FAKE + 2), dict(q=None), dict(q=FAKE + 8), dict(k=FAKE + 2),
    dict(v=None), dict(qts=764), dict(khs=60), dict(vts=-768), dict(kts=1 << 24),
]


@pytest.mark.parametrize("kw", BAD_RAGGED + [dict(out=None), dict(ots=448), dict(ohs=32), dict(lse=FAKE + 2)])
def test_history_attention_rejects(kw):
    h = handle()
    assert rc_of("emb_history_attention", dict(ATT, h=h), {k: (None if k == "h" else v) for k, v in kw.items()}) == INVAL
    E.emb_destroy_history(h)


def test_history_attention_without_buckets_or_tokens():
    h, plain = handle(), handle(buckets=0, exact=0, far=0)
    assert rc_of("emb_history_attention", dict(ATT, h=plain), {}) == INVAL          # a bias without buckets
    assert rc_of("emb_history_attention", dict(ATT, h=h), dict(tokens=0, seqs=0, q=None, off=None)) == OK
    assert E.lib().emb_check_history_error(h, None) == OK and E.lib().emb_check_history_error(None, None) == INVAL
    for x in (h, plain):
        E.emb_destroy_history(x)


BACK_ATT = dict(h=None, tokens=10, q=FAKE, qts=768, qhs=64, k=FAKE, kts=768, khs=64, v=FAKE, vts=768, vhs=64, out=FAKE,
                ots=512, ohs=64, lse=FAKE, dout=FAKE, gts=512, ghs=64, dq=FAKE, dqts=512, dqhs=64, dk=FAKE, dkts=128,
                dkhs=64, dv=FAKE, dvts=128, dvhs=64, off=FAKE, seqs=2, bias=FAKE, ws=FAKE, n=1 << 20, dbias=FAKE, st=None)


@pytest.mark.parametrize("kw,code", [(k, INVAL) for k in BAD_RAGGED] + [
    (dict(lse=None), INVAL), (dict(lse=FAKE + 1), INVAL), (dict(dout=None), INVAL), (dict(gts=1 << 24), INVAL),
    (dict(dq=None), INVAL), (dict(dk=FAKE + 8), INVAL), (dict(dvts=64), INVAL), (dict(dkhs=32), INVAL),
    (dict(ws=None), INVAL), (dict(ws=FAKE + 8), INVAL), (dict(n=100), WS), (dict(dbias=FAKE + 2), INVAL),
])
def test_history_backward_rejects(kw, code):
    h = handle()
    kw = {k: (None if k == "h" else v) for k, v in kw.items()}
    assert rc_of("emb_history_attention_backward", dict(BACK_ATT, h=h), kw) == code
    E.emb_destroy_history(h)


def test_history_workspaces():
    h, kv = handle(), cache()
    f = E.emb_history_attention_workspace_bytes
    assert f(h, 1000, 4) >= 1000 * 8 * 4 and f(h, -1, 4) == 0 and f(h, 10, -1) == 0
    assert E.emb_history_step_workspace_bytes(h, kv, 4, 100) >= 16
    assert E.emb_history_step_workspace_bytes(h, kv, -1, 100) == 0
    E.emb_destroy_history(h)
    E.emb_destroy_kv(kv)


STEP = dict(h=None, kv=None, seqs=4, q=FAKE, qts=512, qhs=64, out=FAKE, ots=512, ohs=64, lens=FAKE, table=FAKE, width=8,
            bias=FAKE, ws=FAKE, n=1 << 24, lse=FAKE, st=None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=0), INVAL), (dict(kv=0), INVAL), (dict(seqs=-1), INVAL), (dict(seqs=1 << 24), INVAL), (dict(q=None), INVAL),
    (dict(q=FAKE + 8), INVAL), (dict(qts=508), INVAL), (dict(out=None), INVAL), (dict(ots=448), INVAL),
    (dict(lens=None), INVAL), (dict(lens=FAKE + 2), INVAL), (dict(table=None), INVAL), (dict(width=-1), INVAL),
    (dict(width=1 << 27), INVAL), (dict(bias=None), INVAL), (dict(bias=FAKE + 1), INVAL), (dict(lse=FAKE + 3), INVAL),
    (dict(ws=None), INVAL), (dict(ws=FAKE + 4), INVAL), (dict(n=8), WS),
])
def test_history_step_rejects(kw, code):
    h, kv = handle(), cache()
    kw = {k: (None if k in ("h", "kv") else v) for k, v in kw.items()}
    assert rc_of("emb_history_step", dict(STEP, h=h, kv=kv), kw) == code
    E.emb_destroy_history(h)
    E.emb_destroy_kv(kv)


@pytest.mark.parametrize("desc,kv,code", [
    (dict(), dict(dim=128), INVAL), (dict(), dict(heads=4), INVAL), (dict(), dict(dtype=E.EMB_F16), DTYPE),
    (dict(), dict(k=FAKE + 2), INVAL), (dict(), dict(slot=68), INVAL), (dict(hq=66, hk=2), dict(), INVAL),
])
def test_history_step_rejects_caches_that_do_not_fit(desc, kv, code):
    h, c = handle(**desc), cache(**kv)
    assert rc_of("emb_history_step", dict(STEP, h=h, kv=c), {}) == code
    E.emb_destroy_history(h)
    E.emb_destroy_kv(c)


def test_history_step_without_sequences():
    h, c = handle(), cache()
    assert rc_of("emb_history_step", dict(STEP, h=h, kv=c), dict(seqs=0, q=None, lens=None, ws=None)) == OK
    E.emb_destroy_history(h)
    E.emb_destroy_kv(c)


def test_history_calls_beyond_one_launch():
    """A launch has less than 2^24 blocks of 256 threads."""
    h, c = handle(), cache()            # 8 query heads, 2 of the cache
    back, step = E.emb_history_attention_workspace_bytes, E.emb_history_step_workspace_bytes
    hq = DESC["hq"]
    most = (1 << 24) // hq - 1
    for seqs, good in ((most, True), (most + 1, False)):
        assert (back(h, 10, seqs) > 0) == good
        if not good:
            assert rc_of("emb_history_attention", dict(ATT, h=h), dict(seqs=seqs)) == INVAL
            assert rc_of("emb_history_attention_backward", dict(BACK_ATT, h=h), dict(seqs=seqs, n=1 << 60)) == INVAL
    most = (1 << 23) // 2 - 1
    assert step(h, c, most, 8) >= 16 and step(h, c, most + 1, 8) == 0
    assert rc_of("emb_history_step", dict(STEP, h=h, kv=c), dict(seqs=most + 1, n=1 << 60)) == INVAL
    E.emb_destroy_history(h)
    E.emb_destroy_kv(c)


def test_history_operands_that_share_memory():
    """What is written must not start where another operand that is read, or written, does."""
    h = handle()
    apart = {n: FAKE + 4096 * i for i, n in enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}
    few = {n: apart[n] for n in ("q", "k", "v", "out")}
    for other in ("k", "v"):
        assert rc_of("emb_history_attention", dict(ATT, h=h, **few), dict(out=apart[other])) == INVAL
    for written in ("dq", "dk", "dv"):
        for other in apart:
            if other != written:
                assert rc_of("emb_history_attention_backward", dict(BACK_ATT, h=h, **apart),
                             {written: apart[other]}) == INVAL
    E.emb_destroy_history(h)
