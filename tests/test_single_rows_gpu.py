"""A packed tensor of one token: its stride is not looked at."""
import pytest
import torch

import split_kv_fd_gb300 as fd

pytestmark = pytest.mark.gpu

STRIDES = [1, -3, 7, 12345, (1 << 44) + 1]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("stride", STRIDES)
def test_prefill(stride):
    q, k, v = (torch.randn(1, h, 128, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want, _ = fd.prefill(q, k, v, cu)
    out = torch.full_like(want, 5)
    ws = torch.empty(fd.workspace_size_extend(1, 1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    st = fd.load().fd_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), cu.data_ptr(), 1, 1, 1, 4, 2, 128,
                              stride, stride, stride, 2, 1, 0.1, out.data_ptr(), 2, None, ws.data_ptr(), ws.numel(), _stream())
    assert st == 0 and torch.equal(out, want)   # one key: its value, whatever the scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stride", STRIDES)
def test_append(stride, dtype):
    k, v = (torch.randn(1, 2, 64, device="cuda").to(dtype) for _ in range(2))
    kp, vp = (torch.zeros(2, 2, 16, 64, dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.tensor([21], dtype=torch.int32, device="cuda")
    st = fd.load().fd_append_paged(k.data_ptr(), v.data_ptr(), slots.data_ptr(), 1, 2, 64, stride, stride,
                                   0 if dtype == torch.float32 else 2, kp.data_ptr(), vp.data_ptr(), 16, 2, _stream())
    assert st == 0
    for x, p in ((k, kp), (v, vp)):
        want = torch.zeros_like(p)
        want[1, :, 5] = x[0]
        assert torch.equal(p, want)
