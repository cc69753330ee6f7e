"""What fd_beam_select promises beside its results: which memory it reads."""
import pytest
import torch

import split_kv_fd_gb300 as fd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def test_finished_beams_are_not_read():
    """4.3 GB of logits, all of their beams finished.  What a call reads passes
    the card's nominal 8 TB/s at most, so its time bounds the share it can have
    read: below a fifth.  (Two reads ahead of the flag would be a quarter, and
    200 us.)"""
    R, W, V = 512, 32, 131072
    x = torch.zeros(R, W, V, dtype=torch.bfloat16, device="cuda")
    scores = -torch.rand(R, W, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    done = torch.ones(R, W, dtype=torch.bool, device="cuda")
    ws = torch.empty(fd.workspace_size_beam(R, W, V, W), dtype=torch.uint8, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    took = []
    for _ in range(10):
        start.record()
        got = fd.beam_select(x, scores, W, finished=done, eos=3, workspace=ws)
        end.record()
        torch.cuda.synchronize()
        took.append(start.elapsed_time(end) * 1e-3)
    want = scores.sort(dim=1, descending=True)
    assert torch.equal(got[0], want.values) and torch.equal(got[1], want.indices.int())
    assert min(took) * 8e12 < 0.2 * x.numel() * 2, f"{min(took) * 1e6:.1f} us"
