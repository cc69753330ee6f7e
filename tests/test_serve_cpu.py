"""The calls around decode without a GPU: bad arguments are refused before
any CUDA call, by the library and by the binding."""
import ctypes

import pytest
import torch

import split_kv_fd_gb300 as fd
from split_kv_fd_gb300 import fd as fdmod
from serve_util import resize_ref

P = ctypes.c_void_p
X = P(4096)      # aligned, never dereferenced
ODD = P(4104)
F32, F16, BF16, E4M3 = 0, 1, 2, 3
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return fdmod.load(build_if_missing=True)


def _prefill(lib, **kw):
    a = dict(q=X, k=X, v=X, cu_q=X, cu_k=X, B=2, tq=10, tk=10, Hq=4, Hkv=2, d=128, qs=512, ks=256, vs=256, dt=BF16, causal=1,
             scale=0.1, out=X, odt=BF16, lse=None, ws=None, nws=0, stream=None)
    a.update(kw)
    return lib.fd_prefill(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(tq=-1), INVALID), (dict(tk=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dt=F32), UNSUPPORTED),
    (dict(dt=E4M3), UNSUPPORTED), (dict(odt=E4M3), UNSUPPORTED), (dict(qs=504), INVALID), (dict(qs=516), INVALID),
    (dict(ks=128), INVALID), (dict(vs=257), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(k=ODD), INVALID),
    (dict(v=None), INVALID), (dict(out=ODD), INVALID), (dict(cu_q=None), INVALID), (dict(cu_k=P(4098)), INVALID),
    (dict(lse=P(4097)), INVALID), (dict(B=0), 0), (dict(tq=0), 0), (dict(Hq=0), 0)])
def test_prefill_refuses(lib, kw, status):
    assert _prefill(lib, **kw) == status


def _extend(lib, fp8=False, **kw):
    a = dict(q=X, qdt=BF16, kp=X, vp=X, ks=X, vsc=X, table=X, cu=X, sl=X, B=2, tq=10, Hq=4, Hkv=2, d=128, qs=512, page=64, width=4,
             pages=9, dt=BF16, scale=0.1, out=X, odt=BF16, lse=None, ws=None, nws=0, stream=None)
    a.update(kw)
    for n in (("dt",) if fp8 else ("qdt", "ks", "vsc")):
        del a[n]
    return (lib.fd_extend_paged_fp8 if fp8 else lib.fd_extend_paged)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(page=0), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=1), UNSUPPORTED), (dict(width=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(page=1 << 20, width=1 << 12), INVALID), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(Hq=5), INVALID), (dict(scale=0.0), INVALID), (dict(table=None), INVALID),
    (dict(sl=None), INVALID), (dict(kp=None), INVALID), (dict(vp=ODD), INVALID), (dict(pages=0), INVALID), (dict(cu=P(4097)), INVALID),
    (dict(B=0), 0), (dict(tq=0), 0)])
def test_extend_refuses(lib, fp8, kw, status):
    assert _extend(lib, fp8, **kw) == status


def test_extend_fp8_refuses(lib):
    assert _extend(lib, True, ks=None) == INVALID
    assert _extend(lib, True, vsc=P(4097)) == INVALID
    assert _extend(lib, True, qdt=F32) == UNSUPPORTED
    assert _extend(lib, False, dt=F32) == UNSUPPORTED


def _resize(lib, **kw):
    a = dict(sl=X, target=X, B=2, table=X, width=4, free=X, count=X, pages=9, page=16, slots=X, pos=X, room=8, cu=X, stream=None)
    a.update(kw)
    return lib.fd_resize_pages(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(width=-1), dict(pages=-1), dict(page=0), dict(room=-1), dict(sl=None),
                                dict(target=None), dict(table=None), dict(free=None), dict(count=None), dict(cu=None),
                                dict(slots=P(4097)), dict(count=P(4098)), dict(page=1 << 20, width=1 << 12),
                                dict(page=1 << 20, pages=1 << 12)])
def test_resize_refuses(lib, kw):
    assert _resize(lib, **kw) == INVALID


def _append(lib, fp8=False, **kw):
    a = dict(k=X, v=X, ks=X, vsc=X, cu=X, slots=X, B=2, T=5, H=2, d=128, kst=256, vst=256, dt=BF16, kp=X, vp=X, page=16, pages=9,
             stream=None)
    a.update(kw)
    if not fp8:
        for n in ("ks", "vsc", "cu", "B"):
            del a[n]
    return (lib.fd_append_paged_fp8 if fp8 else lib.fd_append_paged)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(page=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=1 << 40), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(dt=E4M3), UNSUPPORTED), (dict(kst=128), INVALID), (dict(vst=257), INVALID),
    (dict(k=None), INVALID), (dict(v=ODD), INVALID), (dict(kp=ODD), INVALID), (dict(slots=None), INVALID), (dict(T=0), 0)])
def test_append_refuses(lib, fp8, kw, status):
    assert _append(lib, fp8, **kw) == status


@pytest.mark.parametrize("kw", [dict(B=0), dict(cu=None), dict(ks=None), dict(vsc=P(4097))])
def test_append_fp8_refuses(lib, kw):
    assert _append(lib, True, **kw) == INVALID


def test_workspace_size_refuses(lib):
    for args in ((-1, 8, 4, 2, 128), (1, -8, 4, 2, 128), (1, 8, 4, 0, 128), (1, 8, 5, 2, 128), (1, 8, 4, 2, 96)):
        assert fd.workspace_size_extend(*args) == 0


def test_binding_refuses_host_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    kp = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fd.prefill(q, q, q, i)
    with pytest.raises(ValueError):
        fd.extend_paged(q, kp, kp, i[None], i, i[:1])
    with pytest.raises(ValueError):
        fd.append_paged(q, q, i, kp, kp)
    with pytest.raises(ValueError):
        fd.resize_pages(i, i, i[:, None], i, i[:1], 16)


def test_rows_of_views():
    """What counts as packed rows."""
    x = torch.zeros(6, 10, 64)
    assert fdmod._rows(x, "x") == 640 and fdmod._rows(x[:, 2:5], "x") == 640 and fdmod._rows(x[::2], "x") == 1280
    assert fdmod._rows(x[:1, :3], "x") == 192 and fdmod._rows(x[:0], "x") == 640
    for bad in (x[:, ::2], x[:, :, :32], x.transpose(0, 1), x[:1].expand(6, 10, 64), x[0]):
        with pytest.raises(ValueError):
            fdmod._rows(bad, "x")


def test_the_stack_reference():
    """The tests' own bookkeeping, by hand: pages 3 and 2 come from the top, come back in order."""
    new, table, free, count, slots, pos, cu = resize_ref([0, 16], [17, 0], [[9, 9], [5, 9]], [0, 1, 2, 3, 4, 9], 4, 16)
    assert new == [17, 0] and table == [[5, 3], [5, 9]] and count == 3
    assert slots == [5 * 16 + i for i in range(16)] + [48] and pos == list(range(17)) and cu == [0, 17, 17]
