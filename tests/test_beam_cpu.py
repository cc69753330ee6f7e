"""The beam search calls without a GPU: bad arguments are refused before any
CUDA call, by the library and by the binding."""
import ctypes

import pytest
import torch

import split_kv_fd_gb300 as fd
from split_kv_fd_gb300 import fd as fdmod

P = ctypes.c_void_p
X = P(4096)      # aligned, never dereferenced
F32, F16, BF16, E4M3 = 0, 1, 2, 3
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return fdmod.load(build_if_missing=True)


def _select(lib, **kw):
    a = dict(x=X, dt=BF16, rs=4000, ws=1000, sc=X, fin=X, R=2, W=4, V=1000, K=8, eos=5, osc=X, op=X, ot=X, of=X, wsp=X, n=1 << 30,
             stream=None)
    a.update(kw)
    return lib.fd_beam_select(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(W=0), INVALID), (dict(W=33), INVALID), (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID),
    (dict(V=1, K=5, eos=0), INVALID), (dict(V=1 << 29), INVALID), (dict(R=1 << 30), INVALID), (dict(rs=-1), INVALID),
    (dict(ws=-1), INVALID), (dict(eos=1000), INVALID), (dict(eos=-2), INVALID), (dict(eos=-1), INVALID), (dict(dt=E4M3), UNSUPPORTED),
    (dict(dt=7), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=P(4097)), INVALID), (dict(x=P(4098), dt=F32), INVALID),
    (dict(sc=None), INVALID), (dict(sc=P(4098)), INVALID), (dict(osc=None), INVALID), (dict(op=P(4097)), INVALID),
    (dict(ot=None), INVALID), (dict(R=0), 0)])
def test_select_refuses(lib, kw, status):
    assert _select(lib, **kw) == status


def test_select_workspace_refuses():
    for args in ((-1, 4, 100, 4), (1, 0, 100, 4), (1, 33, 100, 4), (1, 4, 0, 4), (1, 4, 100, 0), (1, 4, 100, 65), (1, 2, 2, 5)):
        assert fd.workspace_size_beam(*args) == 0


def test_binding_refuses():
    x, sc = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        fd.beam_select(x, sc)


def _reorder(lib, **kw):
    a = dict(par=X, R=2, W=4, sl=X, table=X, width=4, free=X, count=X, pages=9, page=16, copies=X, granted=X, ws=X, n=1 << 30, stream=None)
    a.update(kw)
    return lib.fd_reorder_pages(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(W=0), INVALID), (dict(W=33), INVALID), (dict(R=1 << 30, W=2), INVALID), (dict(width=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(page=0), INVALID), (dict(page=1 << 20, width=1 << 12), INVALID),
    (dict(page=1 << 20, pages=1 << 12), INVALID), (dict(par=None), INVALID), (dict(par=P(4098)), INVALID), (dict(sl=None), INVALID),
    (dict(table=None), INVALID), (dict(table=P(4097)), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID),
    (dict(copies=None), INVALID), (dict(granted=P(4098)), INVALID), (dict(ws=None), 3), (dict(n=100), 3), (dict(ws=P(4112)), 3),
    (dict(R=0), 0)])
def test_reorder_refuses(lib, kw, status):
    assert _reorder(lib, **kw) == status


def _copy(lib, **kw):
    a = dict(copies=X, n=4, H=2, d=128, dt=BF16, kp=X, vp=X, page=16, pages=9, stream=None)
    a.update(kw)
    return lib.fd_copy_pages(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(H=-1), INVALID), (dict(page=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=1 << 40), INVALID),
    (dict(H=1 << 25), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(dt=7), UNSUPPORTED),
    (dict(H=1 << 10, page=1 << 20, pages=9), UNSUPPORTED), (dict(copies=None), INVALID), (dict(copies=P(4098)), INVALID),
    (dict(kp=None), INVALID), (dict(vp=P(4104)), INVALID), (dict(n=0), 0), (dict(H=0), 0)])
def test_copy_refuses(lib, kw, status):
    assert _copy(lib, **kw) == status


def test_reorder_workspace_refuses():
    for args in ((-1, 4, 100), (1, 0, 100), (1, 33, 100), (1, 4, -1), (1 << 30, 2, 4)):
        assert fd.workspace_size_reorder(*args) == 0
    assert fd.workspace_size_reorder(0, 4, 100) > 0 and fd.workspace_size_reorder(1, 4, 0) > 0


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fd.reorder_pages(i, i.flatten(), torch.zeros(4, 3, dtype=torch.int32), i[0], i[0, :1], 16)
    kp = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fd.copy_pages(torch.zeros(1, 3, dtype=torch.int32), kp, kp)
