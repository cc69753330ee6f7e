"""Beam search's selection (fd_beam_select) against the definition in float64."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from beam_util import candidates, check_select

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _logits(R, W, V, dtype, seed, pad=0, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(R, W, V + pad, device="cuda", generator=g) * std).to(DT[dtype])
    return x[:, :, :V], -torch.rand(R, W, device="cuda", generator=g) * 8


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,W,V,K,pad", [
    (1, 1, 1, 1, 0), (1, 4, 2, 8, 0), (3, 2, 7, 5, 1), (2, 4, 1000, 8, 0), (5, 3, 1023, 3, 2), (1, 32, 2049, 64, 0), (7, 5, 4097, 10, 3),
    (64, 1, 5000, 2, 0), (2, 8, 32000, 16, 0), (1, 4, 50021, 4, 1), (3, 16, 100003, 32, 5), (40, 8, 8191, 16, 7), (1, 1, 262144, 64, 0),
    (2, 1, 300000, 1, 13)])
def test_against_the_definition(R, W, V, K, pad, dtype):
    x, scores = _logits(R, W, V, dtype, seed=R + W + V, pad=pad)
    same = check_select(fd.beam_select(x, scores, K), x, scores, K)
    assert same >= R * 0.5 - 1 or V < 8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_alignment(dtype):
    """Rows that start at every place of a 16-byte block, and ends likewise."""
    buf = (torch.randn(40000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 4).to(DT[dtype])
    sc = torch.tensor([[-1.0, -1.5]], device="cuda")
    for first in range(9):
        for V in (1, 3, 8, 1024, 1025, 1031, 3000):
            x = buf[first:first + 2 * (V + 3)].view(1, 2, V + 3)[:, :, :V]
            check_select(fd.beam_select(x, sc, min(5, 2 * V)), x, sc, min(5, 2 * V))


def test_strides():
    """Beams that share a row, requests in reverse memory order of beams."""
    x, scores = _logits(4, 3, 777, "bf16", 5)
    one = x[:, :1].expand(4, 3, 777)
    assert one.stride(1) == 0
    check_select(fd.beam_select(one, scores, 6), one, scores, 6)
    turned = x.transpose(0, 1)   # requests next to one another
    check_select(fd.beam_select(turned, scores.t().contiguous(), 4), turned, scores.t().contiguous(), 4)


def test_rows_far_apart():
    """Requests and beams whose distance passes 2^31 elements, by an odd number."""
    V = 3001
    far = 2 ** 31 + 1037
    buf = torch.empty(far + 70000, dtype=torch.bfloat16, device="cuda")
    for R, W, strides in ((2, 3, (far, 20001, 1)), (3, 2, (20001, far, 1))):
        x = buf.as_strided((R, W, V), strides)
        x.copy_((torch.randn(R, W, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(R)) * 3))
        scores = -torch.rand(R, W, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        check_select(fd.beam_select(x, scores, 8), x, scores, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,K,W", [(64, 8, 4), (5000, 32, 4), (70000, 64, 2), (3000, 7, 1)])
def test_ties_go_to_the_lowest_index(V, K, W, dtype):
    """Constant logits and equal beams; a few values only."""
    flat = torch.full((2, W, V), 1.25, dtype=DT[dtype], device="cuda")
    sc = torch.full((2, W), -3.0, device="cuda")
    out, parents, tokens, _ = fd.beam_select(flat, sc, K)
    assert parents.tolist() == [[k // V for k in range(K)]] * 2 and tokens.tolist() == [[k % V for k in range(K)]] * 2
    assert bool((out == out[0, 0]).all()) and abs(float(out[0, 0]) + 3 + math.log(V)) < 1e-5
    g = torch.Generator(device="cuda").manual_seed(V)
    few = torch.randint(0, 3, (1, 1, V), device="cuda", generator=g).to(DT[dtype]).expand(2, W, V).contiguous()
    out, parents, tokens, _ = fd.beam_select(few, sc, K)
    top = (few[0, 0] == 2).nonzero()[:, 0]
    want = [(w, int(t)) for w in range(W) for t in top[:K]][:K]
    assert len(want) == K and [list(zip(p, t)) for p, t in zip(parents.tolist(), tokens.tolist())] == [want] * 2


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rising_and_falling_rows(dtype):
    """The largest values all in one place, in the order that makes the most of them wait."""
    V = 60000
    for x in (torch.linspace(-20, 20, V), torch.linspace(20, -20, V), torch.linspace(-20, 20, V).roll(1500)):
        x = torch.stack([x, x * 0.5, x * 0.25]).to(DT[dtype])[None].cuda()
        sc = torch.tensor([[-1.0, 2.0, 5.0]], device="cuda")
        for K in (1, 9, 64):
            check_select(fd.beam_select(x, sc, K), x, sc, K)


def test_finished_beams():
    x, scores = _logits(6, 4, 3001, "bf16", 8)
    g = torch.Generator(device="cuda").manual_seed(8)
    done = torch.rand(6, 4, device="cuda", generator=g) < 0.5
    done[0], done[1] = True, False
    x = torch.where(done[..., None], math.nan, x)      # what a finished beam's logits hold does not matter
    for eos in (0, 1234, 3000):
        check_select(fd.beam_select(x, scores, 8, finished=done, eos=eos), x, scores, 8, done, eos)
    # all finished: each beam once, then nothing
    out, parents, tokens, over = fd.beam_select(x, scores, 8, finished=torch.ones_like(done), eos=7)
    order = scores.sort(dim=1, descending=True)
    assert torch.equal(out[:, :4], order.values) and torch.equal(parents[:, :4], order.indices.int())
    assert bool((tokens[:, :4] == 7).all()) and bool((tokens[:, 4:] == -1).all()) and bool((out[:, 4:] == -math.inf).all()) and bool(over.all())
    # an eos without finished beams marks what ends
    x, scores = _logits(2, 2, 50, "f32", 9)
    x[:, :, 17] = 30.0
    out, parents, tokens, over = fd.beam_select(x, scores, 2, eos=17)
    assert bool((tokens == 17).all()) and bool(over.all())
    assert not bool(fd.beam_select(x, scores, 2)[3].any())


@pytest.mark.parametrize("V,K,W", [(30, 12, 5), (3000, 64, 6), (90000, 20, 32)])
def test_finished_beams_among_many_equal_ones(V, K, W):
    """Rows that leave more candidates than fit the short list, with finished beams between, ahead and behind."""
    x = torch.full((3, W, V), -0.5, device="cuda")
    x[1] = torch.arange(V, device="cuda") % 5
    x[2, :, : V // 2] = -math.inf
    base = -1.0 - math.log(V)
    scores = torch.full((3, W), -1.0, device="cuda")
    done = torch.zeros(3, W, dtype=torch.bool, device="cuda")
    done[:, 1], done[:, W - 1] = True, True
    scores[:, 1], scores[:, W - 1] = base + 0.01, -50.0
    for eos in (0, V - 1):
        check_select(fd.beam_select(x, scores, K, finished=done, eos=eos), x, scores, K, done, eos)


def test_few_continuations():
    """Beams without a score, masked tokens, rows that the mask leaves empty."""
    x, scores = _logits(5, 3, 900, "f16", 10)
    x = x.clone()
    scores[0] = torch.tensor([-math.inf, -2.0, -math.inf])
    scores[1] = torch.tensor([math.nan, math.inf, -math.inf])     # nothing at all
    x[2, 0], x[2, 1] = -math.inf, math.nan                        # two rows empty
    x[3] = -math.inf
    x[3, 1, 5], x[3, 2, 899] = 0.0, -3.0                          # one token each
    x[4, :, 10:] = torch.finfo(torch.float16).min                 # masks of the type's lowest value
    for K in (1, 4, 20):
        got = fd.beam_select(x, scores, K)
        check_select(got, x, scores, K)
    assert got[1][1].tolist() == [-1] * 20 and got[1][3, 2:].tolist() == [-1] * 18
    assert got[2][3, :2].tolist() == [5, 899] or got[2][3, :2].tolist() == [899, 5]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_values_that_are_not_finite(dtype):
    x, scores = _logits(6, 2, 2500, dtype, 12)
    x = x.clone()
    x[0, 0, 100::7] = math.nan
    x[1, 0, 2400] = math.inf                                      # counts as the largest finite value
    x[2, 1, [3, 1700]] = math.inf
    x[3, :, ::2] = -math.inf
    x[4, 0, :] = torch.finfo(DT[dtype]).min                       # a whole row of the lowest value: uniform
    x[5, 0, 0], x[5, 0, 2499], x[5, 1, 5] = math.nan, math.inf, -math.inf
    check_select(fd.beam_select(x, scores, 6), x, scores, 6)
    got = fd.beam_select(x[1:2], scores[1:2] * 0, 3)
    assert got[1][0, 0] == 0 and got[2][0, 0] == 2400 and float(got[0][0, 0]) == 0.0


def test_scores_far_from_zero():
    """What the sum of a score and a logit would cut off decides."""
    V = 4000
    x = torch.zeros(1, 2, V, device="cuda")
    x[0, 0] = -torch.arange(V, device="cuda") * 2.0 ** -18
    x[0, 1] = -torch.arange(V, device="cuda") * 2.0 ** -18
    sc = torch.tensor([[-50000.0, -90000.0]], device="cuda")
    out, parents, tokens, _ = fd.beam_select(x, sc, 32)
    assert tokens[0].tolist() == list(range(32)) and not bool(parents.any())
    for scale in (1e-3, 1.0, 1e4, 1e30):
        x, sc = _logits(2, 4, 5000, "f32", 31)
        x = x * scale
        check_select(fd.beam_select(x, sc, 8), x, sc, 8)


def test_the_sum_is_close_to_its_value():
    """Rows whose logarithm of the sum a float32 sum in one chain would miss."""
    V = 262144
    for x in (torch.zeros(V), torch.linspace(-1, 0, V), torch.where(torch.arange(V) % 4096 == 0, 0.0, -9.0)):
        x = x.cuda().view(1, 1, V)
        sc = torch.zeros(1, 1, device="cuda")
        out = fd.beam_select(x, sc, 1)[0]
        want = candidates(x, sc).amax()
        assert abs(float(out) - float(want)) < 2e-6


def test_same_from_call_to_call_and_between_equal_beams():
    x, scores = _logits(8, 4, 40000, "bf16", 14)
    x[:, 2], scores[:, 2] = x[:, 0], scores[:, 0]
    first = fd.beam_select(x, scores, 16)
    for _ in range(20):
        for a, b in zip(first, fd.beam_select(x, scores, 16)):
            assert torch.equal(a, b)
    out, parents, tokens, _ = (t.cpu() for t in first)
    for r in range(8):   # a copy comes right behind, at the same score
        for k in (parents[r] == 0).nonzero()[:, 0].tolist():
            twin = ((parents[r] == 2) & (tokens[r] == tokens[r, k])).nonzero()[:, 0].tolist()
            assert all(out[r, t] == out[r, k] for t in twin)


def test_streams_workspaces_and_graphs():
    x, scores = _logits(4, 4, 9000, "f32", 15)
    want = fd.beam_select(x, scores, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [fd.beam_select(x, scores, 8, stream=side) for _ in range(3)][-1]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    ws = torch.empty(fd.workspace_size_beam(4, 4, 9000, 8), dtype=torch.uint8, device="cuda").fill_(0xff)
    torch.cuda.synchronize()
    graphs = []
    for num in (8, 3):   # two graphs on one workspace, replayed one behind the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fd.beam_select(x, scores, num, workspace=ws)
        graphs.append((g, out, num))
    x.copy_(_logits(4, 4, 9000, "f32", 16)[0])
    for g, _, _ in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for _, out, num in graphs:
        check_select(out, x, scores, num)


def test_refusals():
    x, scores = _logits(2, 3, 100, "f32", 17)
    done = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    for kw in (dict(num=0), dict(num=65), dict(num=-1), dict(eos=100), dict(eos=-2), dict(finished=done),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, fd.FDError)):
            fd.beam_select(x, scores, **kw)
    with pytest.raises(fd.FDError):
        fd.beam_select(x[:, :, :2], scores, 7)
    wide = torch.zeros(1, 33, 4, device="cuda")
    with pytest.raises(fd.FDError):
        fd.beam_select(wide, torch.zeros(1, 33, device="cuda"), 2)
    empty = fd.beam_select(x[:0], scores[:0])
    assert [t.shape for t in empty] == [(0, 3)] * 4
