"""Refusals of layer norm and dropout (CPU): every bad call is turned away with its status code and a message before
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
