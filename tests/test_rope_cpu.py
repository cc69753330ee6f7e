"""The rotating appends without a GPU: bad arguments are refused before any
CUDA call, by the library and by the binding."""
import ctypes

import pytest
import torch

import split_kv_fd_gb300 as fd
from split_kv_fd_gb300 import fd as fdmod

P = ctypes.c_void_p
X = P(4096)      # aligned, never dereferenced
ODD = P(4104)
F32, F16, BF16, E4M3 = 0, 1, 2, 3
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return fdmod.load(build_if_missing=True)


def _rope(lib, fp8=False, **kw):
    a = dict(q=X, k=X, v=X, ks=X, vsc=X, cu=X, slots=X, pos=X, rope=X, far=100, rot=128, pairs=0, B=2, T=5, Hq=8, H=2, d=128,
             qst=1024, kst=256, vst=256, dt=BF16, qo=X, qost=1024, kp=X, vp=X, page=16, pages=9, stream=None)
    a.update(kw)
    if not fp8:
        for n in ("ks", "vsc", "cu", "B"):
            del a[n]
    return (lib.fd_append_rope_paged_fp8 if fp8 else lib.fd_append_rope_paged)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=-1), INVALID), (dict(Hq=-1), INVALID), (dict(page=0), INVALID),
    (dict(pages=-1), INVALID), (dict(pages=1 << 40), INVALID), (dict(far=-1), INVALID), (dict(Hq=1 << 24), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(dt=E4M3), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=8), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED), (dict(kst=128), INVALID),
    (dict(vst=257), INVALID), (dict(qst=1000), INVALID), (dict(qst=1028), INVALID), (dict(qost=512), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(qo=None), INVALID), (dict(qo=ODD), INVALID), (dict(k=None), INVALID),
    (dict(v=ODD), INVALID), (dict(kp=ODD), INVALID), (dict(vp=None), INVALID), (dict(slots=None), INVALID),
    (dict(pos=None), INVALID), (dict(pos=P(4098)), INVALID), (dict(rope=None), INVALID), (dict(rope=ODD), INVALID),
    (dict(T=0), 0)])
def test_refuses(lib, fp8, kw, status):
    assert _rope(lib, fp8, **kw) == status


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=(1 << 30) + 1), dict(cu=None), dict(ks=None), dict(vsc=P(4097))])
def test_fp8_refuses(lib, kw):
    assert _rope(lib, True, **kw) == INVALID


def test_status_has_a_name(lib):
    assert fdmod.status_str(9).startswith("FD_ERR_BAD_INDEX")


def test_binding_refuses_host_tensors():
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    kp = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    s = torch.ones(1, 2)
    with pytest.raises(ValueError):
        fd.append_rope_paged(k, k, i, i, torch.zeros(8, 64), kp, kp)
    with pytest.raises(ValueError):
        fd.append_rope_paged_fp8(k, k, s, s, i[:2], i, i, torch.zeros(8, 64), kp.to(torch.uint8), kp.to(torch.uint8))


def test_binding_checks_before_the_call():
    """What the arguments' checks themselves say, on host tensors."""
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    kp = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    rope = torch.zeros(8, 64)

    def args(rope=rope, positions=i, q=None, q_out=None):
        return fdmod._rope_args(k, k, i, positions, rope, kp, kp, q, q_out, False, None)

    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    assert args()[2][:4] == (4, 0, 2, 64) and args(q=q)[2][1] == 6
    for bad in (dict(rope=rope.double()), dict(rope=rope[0]), dict(rope=rope.t()), dict(positions=i[:3]), dict(positions=i.long()),
                dict(q_out=q), dict(q=q.float()), dict(q=q[:3]), dict(q=q[:, :, :32]), dict(q=q, q_out=q[:, :5]),
                dict(q=q, q_out=q.float())):
        with pytest.raises(ValueError):
            args(**bad)
