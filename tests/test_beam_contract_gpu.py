"""What fd_beam_select promises beside its results: which memory it reads, what
its scores depend on, and where a continuation ends to be one."""
import math

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


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 32003), (torch.float32, 50021)])
def test_a_request_in_other_batches_and_places(dtype, V):
    """The same request alone, among others and at every distance from a 16-byte
    boundary: each beam's tokens in the same order, scores within twice the sums'
    error; the same call again, the same bits."""
    W, K = 4, 8
    g = torch.Generator(device="cuda").manual_seed(V)
    one = (torch.randn(1, W, V, device="cuda", generator=g) * 3).to(dtype)
    score = -torch.rand(1, W, device="cuda", generator=g)
    per = 16 // one.element_size()
    first, tol = None, 2 * (90 + 2.25 * math.log(V)) * 2.0 ** -24
    for R, off in ((1, 0), (150, 0), *((1 + o % 3, o) for o in range(1, per))):
        buf = torch.randn(R * W * V + per, device="cuda", generator=g).to(dtype)
        x = buf[off:off + R * W * V].view(R, W, V)
        x[R - 1] = one[0]
        s = score.expand(R, W).contiguous()
        got, again = fd.beam_select(x, s, K), fd.beam_select(x, s, K)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        out, parents, tokens, _ = (t[R - 1].cpu() for t in got)
        rows = {w: tokens[parents == w].tolist() for w in range(W)}
        if first is None:
            first = out, rows
        for w in range(W):   # (a beam may have one more or less among the K where two are near)
            n = min(len(rows[w]), len(first[1][w]))
            assert rows[w][:n] == first[1][w][:n]
        assert float((out - first[0]).abs().max()) <= tol + 2.0 ** -23 * float(out.abs().max())


def test_distances_that_float32_does_not_hold():
    """A logit further below the beam's largest than float32 reaches is no continuation, whatever the score."""
    x = torch.tensor([[[3e38, -3e38, 2e38], [1.0, 1.0, 1.0]]], device="cuda")
    for score in (3e38, 0.0, -3e38):
        out, parents, tokens, over = fd.beam_select(x, torch.tensor([[score, -math.inf]], device="cuda"), 4)
        n = 2 if score > -2e38 else 1
        assert tokens.tolist() == [[0, 2][:n] + [-1] * (4 - n)] and over.tolist() == [[False] * n + [True] * (4 - n)]
        assert float(out[0, 0]) == torch.tensor(score).item()
