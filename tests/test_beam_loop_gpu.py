"""Beam search over a paged cache, the calls together as a serving loop uses
them: prompts appended with the rotation, every request's state to its beams,
then steps of decode, selection, reordering, growth and append, with two
layers.  The tokens of every beam are kept beside, and its attention is held to
the definition in float64 over its own history."""
import math
import random

import pytest
import torch

import split_kv_fd_gb300 as fd
from beam_util import check_select
from serve_util import attend, check, pack_offsets

pytestmark = pytest.mark.gpu

LAYERS, VOCAB, FAR = 2, 503, 512


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


class Model:
    """Projections of a token in each layer by a table, and logits from what the layers attend to."""

    def __init__(self, Hq, Hkv, d, rot, pairs, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.rot, self.pairs = Hq, Hkv, d, rot, pairs
        self.qkv = [torch.randn(VOCAB, Hq + 2 * Hkv, d, device="cuda", generator=g).to(dtype) for _ in range(LAYERS)]
        self.head = torch.randn(Hq * d, VOCAB, device="cuda", generator=g) * (4 / math.sqrt(Hq * d))
        a = torch.arange(FAR, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / -rot)
        self.rope = torch.cat([a.cos(), a.sin()], 1).float()

    def split(self, layer, tokens):
        return self.qkv[layer][tokens].split([self.Hq, self.Hkv, self.Hkv], dim=1)

    def logits(self, outs):
        return torch.stack([o.float().flatten(1) for o in outs]).sum(0) @ self.head

    def turn(self, x, positions):
        """x [n, H, d] turned in float32 and rounded, as the append keeps it."""
        row, half = self.rope[positions][:, None], self.rot // 2
        at = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.pairs else (slice(0, half), slice(half, self.rot))
        f = x.float()
        y = f.clone()
        y[..., at[0]] = f[..., at[0]] * row[..., :half] - f[..., at[1]] * row[..., half:]
        y[..., at[1]] = f[..., at[1]] * row[..., :half] + f[..., at[0]] * row[..., half:]
        return y.to(x.dtype)

    def attention(self, layer, tokens):
        """The last token's attention over its history, the reference of serve_util.check."""
        q, k, v = self.split(layer, torch.tensor(tokens, device="cuda"))
        at = torch.arange(len(tokens), device="cuda")
        return attend(self.turn(q, at)[-1:], self.turn(k, at), v)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("R,W,page,Hq,Hkv,d,rot,pairs,dtype", [
    (3, 4, 16, 8, 2, 64, 64, False, torch.bfloat16), (2, 5, 32, 4, 4, 128, 48, True, torch.float16)])
def test_beam_search(R, W, page, Hq, Hkv, d, rot, pairs, dtype, captured):
    steps, B, width = 24, R * W, 6
    m = Model(Hq, Hkv, d, rot, pairs, dtype, seed=R)
    rng = random.Random(R)
    eos = 11
    prompts = [[rng.randrange(20, VOCAB) for _ in range(rng.randint(3, 50))] for _ in range(R)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    pool = B * width
    free, count = torch.randperm(pool, device="cuda").to(torch.int32), i32([pool])
    table, lens = torch.zeros(B, width, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    layers = [tuple(torch.full((pool, Hkv, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2)) for _ in range(LAYERS)]

    # the prompts into the first beams' pages; their last tokens' logits choose the first step's
    target = [len(prompts[r]) if w == 0 else 0 for r in range(R) for w in range(W)]
    T = sum(target)
    slots, positions = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = fd.resize_pages(lens, i32(target), table, free, count, page, slots=slots, positions=positions)
    assert cu.tolist() == pack_offsets(target).tolist()
    packed = torch.tensor([t for p in prompts for t in p], device="cuda")
    outs = []
    for layer, (kp, vp) in enumerate(layers):
        q, k, v = m.split(layer, packed)
        q = fd.append_rope_paged(k, v, slots, positions, m.rope, kp, vp, q=q, interleaved=pairs)
        outs.append(fd.extend_paged(q, kp, vp, table, cu, lens)[0])
    last = (torch.tensor([len(p) for p in prompts]).cumsum(0) - 1).cuda()
    logits = m.logits([o[last] for o in outs])[:, None].expand(R, W, VOCAB).contiguous()
    scores = torch.full((R, W), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(R, W, dtype=torch.bool, device="cuda")
    beams = [[list(p) for _ in range(W)] for p in prompts]

    # a step's buffers, as a captured one keeps them
    tokens = torch.zeros(B, dtype=torch.int64, device="cuda")
    slots, positions = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    copies, granted = torch.zeros(B, 3, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    kept = [torch.zeros(B, Hq, d, dtype=dtype, device="cuda") for _ in range(LAYERS)]
    kept_lse = [torch.zeros(B, Hq, device="cuda") for _ in range(LAYERS)]
    parents, picked = (torch.zeros(R, W, dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        got = fd.beam_select(logits, scores, W, finished=done, eos=eos)
        for to, x in zip((scores, parents, picked, done), got):
            to.copy_(x)
        fd.reorder_pages(parents, lens, table, free, count, page, copies=copies, granted=granted)
        for kp, vp in layers:
            fd.copy_pages(copies, kp, vp)
        # a beam that lives takes its token's place; the tokens are packed, a beam behind the other
        goes = ~done.flatten()
        fd.resize_pages(lens, lens + goes.int(), table, free, count, page, slots=slots, positions=positions, cu_new=cu)
        tokens.copy_(picked.flatten().clamp(min=0))
        order = torch.argsort((~goes).int(), stable=True)
        now = tokens[order]
        new = []
        for layer, (kp, vp) in enumerate(layers):
            q, k, v = m.split(layer, now)
            q = fd.append_rope_paged(k, v, slots, positions, m.rope, kp, vp, q=q, interleaved=pairs)
            mine = torch.zeros(B, Hq, d, dtype=dtype, device="cuda").index_copy_(0, order, q)
            out, lse = fd.decode_gqa_paged(mine, kp, vp, table, lens)
            kept[layer].copy_(out)
            kept_lse[layer].copy_(lse)
            new.append(out)
        logits.copy_(m.logits(new).view(R, W, VOCAB))

    graph = None
    ended = 0
    for i in range(steps):
        before = logits.clone(), scores.clone(), done.clone()
        if not captured or i == 0:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        check_select((scores, parents, picked, done), *before[:2], W, before[2], eos)
        assert bool(granted.all()) and fd.device_status() == 0
        par, tok, over = parents.tolist(), picked.tolist(), done.tolist()
        beams = [[beams[r][par[r][w]] + ([] if over[r][w] else [tok[r][w]]) for w in range(W)] for r in range(R)]
        assert lens.tolist() == [len(b) for bs in beams for b in bs]
        ended = sum(map(sum, over))
        # each beam's attention over its own history
        for b in range(B):
            r, w = divmod(b, W)
            if over[r][w]:
                continue
            for layer in range(LAYERS):
                check(kept[layer][b:b + 1], kept_lse[layer][b:b + 1], m.attention(layer, beams[r][w]), dtype, len(beams[r][w]),
                      f"step {i}, beam {b}, layer {layer}")
        # pages are named by one request, or free
        named = [{p for w in range(W) for p in table[r * W + w, : -(-len(beams[r][w]) // page)].tolist()} for r in range(R)]
        assert sum(map(len, named)) + int(count) == len(set().union(*named, free[: int(count)].tolist())) == pool
    assert ended < B
    # the requests end
    fd.reorder_pages(torch.full_like(parents, -1), lens, table, free, count, page)
    assert int(count) == pool and sorted(free.tolist()) == list(range(pool)) and not bool(lens.any())


def test_beams_over_an_e4m3_cache():
    """A prompt, its state to the beams, a token each and another choice, in
    E4M3 pages: what each beam reads through its table is its own history,
    turned and rounded, and its attention that over the same bytes in a row."""
    R, W, Hq, Hkv, d, page, width = 2, 3, 8, 2, 128, 16, 6
    B = R * W
    m = Model(Hq, Hkv, d, 96, False, torch.bfloat16, seed=5)
    rng = random.Random(5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    # the beams of a request read the same bytes, with the same scales
    scale = [(torch.rand(R, Hkv, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)) / 50 + 0.01).repeat_interleave(W, 0)
             .contiguous() for i in (1, 2)]
    pool = B * width
    free, count = torch.arange(pool, device="cuda").to(torch.int32), i32([pool])
    table, lens = torch.zeros(B, width, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((pool, Hkv, page, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))   # NaN

    def write(target, tokens):
        T = len(tokens)
        slots, positions = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
        cu = fd.resize_pages(lens, i32(target), table, free, count, page, slots=slots, positions=positions)
        q, k, v = m.split(0, torch.tensor(tokens, device="cuda"))
        return fd.append_rope_paged_fp8(k, v, *scale, cu, slots, positions, m.rope, kp.view(torch.float8_e4m3fn),
                                        vp.view(torch.float8_e4m3fn), q=q)

    beams = [[rng.randrange(VOCAB) for _ in range(n)] for n in (37, 16)]
    write([len(beams[0]), 0, 0, len(beams[1]), 0, 0], beams[0] + beams[1])
    beams = [[list(b)] * W for b in beams]
    for parents in ([[0, 0, 0]] * R, [[2, 0, 0], [1, 1, 2]], [[0, 1, 1], [2, 2, 0]]):
        copies, granted = fd.reorder_pages(i32(parents), lens, table, free, count, page)
        fd.copy_pages(copies, kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn))
        assert bool(granted.all())
        beams = [[beams[r][p] + [rng.randrange(VOCAB)] for p in parents[r]] for r in range(R)]
        q = write([len(b) for bs in beams for b in bs], [b[-1] for bs in beams for b in bs])
        out, lse = fd.decode_gqa_paged_fp8(q, kp, vp, *scale, table, lens)
        for b in range(B):
            tokens = beams[b // W][b % W]
            n = len(tokens)
            at = torch.arange(n, device="cuda")
            got = [x[table[b, at // page].long(), :, at % page] for x in (kp, vp)]
            _, k, v = m.split(0, torch.tensor(tokens, device="cuda"))
            row, half = m.rope[at][:, None], 48
            f = k.float()
            y = f.clone()
            y[..., :half] = f[..., :half] * row[..., :half] - f[..., half:96] * row[..., half:]
            y[..., half:96] = f[..., half:96] * row[..., :half] + f[..., :half] * row[..., half:]
            for x, have, sc in ((y, got[0], scale[0]), (v.float(), got[1], scale[1])):
                want = (x / sc[b][None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                assert torch.equal(have, want), f"beam {b}"
            plain = [x.transpose(0, 1).contiguous()[None] for x in got]   # [1, Hkv, n, d]
            o, s = fd.decode_gqa_fp8(q[b:b + 1].contiguous(), *plain, scale[0][b:b + 1].contiguous(), scale[1][b:b + 1].contiguous())
            # both are E4M3 decode on the tensor cores over the same bytes, in 16-bit or in 8-bit parts close to
            # float32: a step of the output's type, 2^-8, of the largest value there may be
            top = float((got[1].view(torch.float8_e4m3fn).float().abs().amax() * scale[1][b].amax()))
            assert float((out[b] - o[0]).float().abs().max()) <= 2.0 ** -8 * top and float((lse[b] - s[0]).abs().max()) <= 1e-3
