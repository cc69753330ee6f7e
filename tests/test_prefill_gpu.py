"""Attention over packed prompts on the GPU (fd_prefill) against the
definition in float64, element by element, at tolerances derived in
serve_util: lengths from 0 and 1 to thousands, every kind of head group,
strided views, fewer keys than queries, values that are not finite where
nobody looks."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import attend, check, half_step, pack_offsets

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _packed(lens, H, d, dtype, seed, pad=0, fill=math.nan):
    """Rows of all sequences, `pad` rows of `fill` before and behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(sum(lens) + 2 * pad, H, d, device="cuda", generator=g).to(DT[dtype])
    if pad:
        x[:pad] = fill
        x[-pad:] = fill
    return x


def _run(lens_q, lens_k, Hq, Hkv, d, dtype, causal=True, seed=0, out_dtype=torch.float32, scale=None):
    pad = 3
    q = _packed(lens_q, Hq, d, dtype, seed, pad)
    k, v = (_packed(lens_k, Hkv, d, dtype, seed + i, pad) for i in (1, 2))
    cq, ck = ((pack_offsets(x) + pad).cuda() for x in (lens_q, lens_k))
    out = torch.full((q.shape[0], Hq, d), 5.0, dtype=out_dtype, device="cuda")
    lse = torch.full((q.shape[0], Hq), 5.0, device="cuda")
    fd.prefill(q, k, v, cq, ck, causal=causal, scale=scale, out=out, lse=lse)
    assert bool((out[:pad] == 5).all() and (out[q.shape[0] - pad:] == 5).all()), "rows of no sequence are not written"
    assert bool((lse[:pad] == 5).all() and (lse[q.shape[0] - pad:] == 5).all())
    for b in range(len(lens_q)):
        rows = slice(int(cq[b]), int(cq[b + 1]))
        keys = slice(int(ck[b]), int(ck[b + 1]))
        ref = attend(q[rows], k[keys], v[keys], causal, scale)
        check(out[rows], lse[rows], ref, DT[dtype], lens_k[b], f"sequence {b} ({lens_q[b]}, {lens_k[b]})")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (8, 2), (3, 1), (14, 2), (16, 1)])
def test_groups(dtype, d, Hq, Hkv):
    lens = [1, 0, 130, 17, 300]
    _run(lens, lens, Hq, Hkv, d, dtype, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (100, 1), (130, 1), (300, 2)])
def test_large_groups(Hq, Hkv):
    _run([70, 1, 5], [70, 1, 5], Hq, Hkv, 64, "bf16", seed=Hq)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 511, 513, 1025, 2047])
def test_lengths(n):
    _run([n], [n], 4, 2, 128, "bf16", seed=n)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens_q,lens_k", [([5, 40], [200, 1]), ([200, 64], [5, 64]), ([1, 1, 1], [1000, 0, 300]),
                                           ([300, 130], [0, 0]), ([129], [128]), ([128], [129]), ([600], [257])])
def test_queries_and_keys_of_different_lengths(causal, lens_q, lens_k):
    """More queries than keys leave the first rows empty: out 0, lse -inf."""
    _run(lens_q, lens_k, 6, 2, 128, "f16", causal=causal, seed=len(lens_q))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_output_types(out_dtype):
    _run([90, 222], [90, 222], 8, 2, 128, "bf16", out_dtype=out_dtype, seed=4)


@pytest.mark.parametrize("scale", [1e-6, 0.02, 1.0, 3.0])
def test_scales(scale):
    _run([333], [333], 4, 2, 64, "bf16", scale=scale, seed=5)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    _run(lens, lens, 4, 2, 64, "bf16", seed=6)


def test_long_prompt():
    """A prompt longer than one tile by far, next to short ones."""
    _run([1, 5003, 77], [1, 5003, 77], 4, 1, 128, "bf16", seed=7)


def test_views_of_a_fused_projection():
    Hq, Hkv, d, lens = 8, 2, 128, [70, 200]
    qkv = torch.randn(270, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = pack_offsets(lens).cuda()
    a = fd.prefill(q, k, v, cu)
    b = fd.prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_growing_scores():
    """Later keys with ever larger scores: the running maximum moves all the time."""
    n, d = 1500, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(d, device="cuda", generator=g)
    k = (u * torch.linspace(-3, 3, n, device="cuda")[:, None])[:, None].to(torch.bfloat16)
    v = torch.randn(n, 1, d, device="cuda", generator=g).to(torch.bfloat16)
    q = u.expand(n, 1, d).to(torch.bfloat16).contiguous()
    cu = pack_offsets([n]).cuda()
    out, lse = fd.prefill(q, k, v, cu, out_dtype=torch.float32)
    check(out, lse, attend(q, k, v), torch.bfloat16, n, "ascending")
    k = k.flip(0).contiguous()
    out, lse = fd.prefill(q, k, v, cu, out_dtype=torch.float32)
    check(out, lse, attend(q, k, v), torch.bfloat16, n, "descending")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_other_sequences_values_do_not_leak(bad):
    """K and V of one sequence hold nothing finite; its neighbours' results are those without it."""
    lens = [100, 60, 200]
    q, k, v = (_packed(lens, 4, 128, "bf16", s) for s in (1, 2, 3))
    cu = pack_offsets(lens).cuda()
    want = fd.prefill(q, k, v, cu)
    k[100:160] = bad
    v[100:160] = bad
    got = fd.prefill(q, k, v, cu)
    for w, x in zip(want, got):
        assert torch.equal(w[:100], x[:100]) and torch.equal(w[160:], x[160:])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_unseen_keys_do_not_leak(bad):
    """A key that is not finite touches only the queries that see it."""
    n = 300
    q, k, v = (_packed([n], 2, 64, "f16", s) for s in (4, 5, 6))
    cu = pack_offsets([n]).cuda()
    want = fd.prefill(q, k, v, cu)
    k[170] = bad
    got = fd.prefill(q, k, v, cu)
    assert torch.equal(want[0][:170], got[0][:170]) and torch.equal(want[1][:170], got[1][:170])


def test_same_call_twice_same_bits():
    lens = [1000, 31, 2000, 400]
    q, k, v = (_packed(lens, h, 128, "bf16", h) for h in (8, 2, 2))
    cu = pack_offsets(lens).cuda()
    a = fd.prefill(q, k, v, cu)
    for _ in range(3):
        b = fd.prefill(q, k, v, cu)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_without_lse_and_empty_batches():
    q = torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16)
    cu = pack_offsets([8]).cuda()
    out, lse = fd.prefill(q, q, q, cu, return_lse=False)
    assert lse is None
    assert torch.equal(out, fd.prefill(q, q, q, cu)[0])
    e = q[:0]
    out, lse = fd.prefill(e, e, e, pack_offsets([0, 0]).cuda())
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    kept = torch.full((8, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fd.prefill(q, q, q, pack_offsets([0, 0]).cuda(), out=kept)
    assert bool((kept == 3).all())
    out, lse = fd.prefill(q, e, e, cu, pack_offsets([0]).cuda())
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_offsets_that_do_not_ascend_are_reported():
    q = torch.randn(64, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 40, 10, 90], dtype=torch.int32, device="cuda")
    fd.prefill(q, q, q, cu)
    assert fd.device_status() == 8
    cu = torch.tensor([0, 64] * 40 + [64], dtype=torch.int32, device="cuda")   # as if 40 sequences shared the rows
    fd.prefill(q, q, q, cu)
    assert fd.device_status() == 8


def test_captured_graphs_with_new_lengths():
    """Two graphs of one call each, replayed in turn after writing new
    offsets: neither disturbs the other."""
    T, Hq, Hkv, d = 700, 8, 2, 128
    sets = []
    for seed in (1, 2):
        q, k, v = (_packed([T], h, d, "bf16", seed * 10 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        cu = pack_offsets([T, 0, 0]).cuda()
        out = torch.zeros(T, Hq, d, dtype=torch.float32, device="cuda")
        lse = torch.zeros(T, Hq, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fd.prefill(q, k, v, cu, out=out, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fd.prefill(q, k, v, cu, out=out, lse=lse)
        sets.append((q, k, v, cu, out, lse, graph))
    for lens in ([700, 0, 0], [1, 300, 399], [256, 256, 188], [0, 3, 10]):
        for q, k, v, cu, out, lse, graph in sets:
            cu.copy_(pack_offsets(lens))
            graph.replay()
        for q, k, v, cu, out, lse, graph in sets:
            at = 0
            for n in lens:
                rows = slice(at, at + n)
                at += n
                if n:
                    check(out[rows], lse[rows], attend(q[rows], k[rows], v[rows]), torch.bfloat16, n, f"{lens}")


def test_two_streams_at_once():
    q, k, v = (_packed([3000], h, 128, "bf16", h) for h in (8, 2, 2))
    cu = pack_offsets([3000]).cuda()
    want = fd.prefill(q, k, v, cu)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            got.append(fd.prefill(q, k, v, cu, stream=s))
    torch.cuda.synchronize()
    for o, z in got:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_memory_of_the_stream_that_works():
    """What a call on another stream allocates is not what the current
    stream has given back but still writes to."""
    q, k, v = (_packed([500], h, 128, "bf16", h) for h in (8, 2, 2))
    cu = pack_offsets([500]).cuda()
    want = fd.prefill(q, k, v, cu)
    busy = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want]
    for _ in range(6):
        busy = busy @ busy
    for t in late:
        t.fill_(7)
    del late, t
    out, lse = fd.prefill(q, k, v, cu, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_single_row_has_no_stride():
    q, k, v = (_packed([1], h, 128, "bf16", h) for h in (4, 2, 2))
    cu = pack_offsets([1]).cuda()
    want, _ = fd.prefill(q, k, v, cu)
    out = torch.empty_like(want)
    ws = torch.empty(fd.workspace_size_extend(1, 1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    for stride in (0, -64, 1 << 44):
        out.fill_(5)
        st = fd.load().fd_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), cu.data_ptr(), 1, 1, 1, 4, 2, 128,
                                  stride, stride, stride, 2, 1, 0.1, out.data_ptr(), 2, None, ws.data_ptr(), ws.numel(),
                                  torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(out, want)   # one key: its value, whatever the scale


def test_long_rows_past_32_bits():
    """Tokens so far apart that element offsets pass 2^31 (a wide view)."""
    H, d, T = 2, 64, 40
    wide = torch.empty(T, 1 << 26, dtype=torch.bfloat16, device="cuda")
    q = wide[:, : H * d].view(T, H, d)
    k = wide[:, 4096:4096 + H * d].view(T, H, d)
    v = wide[:, (1 << 25):(1 << 25) + H * d].view(T, H, d)
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (q, k, v):
        t.copy_(torch.randn(T, H, d, device="cuda", generator=g))
    cu = pack_offsets([T]).cuda()
    a = fd.prefill(q, k, v, cu)
    b = fd.prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tolerance_counts_half_steps():
    """The tolerance is the one that the types give."""
    assert half_step(torch.bfloat16) == 2.0 ** -8 and half_step(torch.float16) == 2.0 ** -11
