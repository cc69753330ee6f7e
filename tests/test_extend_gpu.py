"""Attention of new tokens over a paged cache on the GPU (fd_extend_paged,
_fp8) against the definition in float64 on the gathered rows.  Unused pages
and rows behind each length are NaN, unused table entries name no page."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import attend, check, pack_offsets, paged_cache

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _run(new, lens, Hq, Hkv, d, page, dtype="bf16", seed=0, out_dtype=torch.float32, max_pages=None):
    kp, vp, table, ks, vs = paged_cache(lens, page, Hkv, d, DT[dtype], seed, max_pages=max_pages)
    g = torch.Generator().manual_seed(seed + 99)
    q = torch.randn(sum(new) + 2, Hq, d, generator=g).to(DT[dtype]).cuda()
    out = torch.full(q.shape, 5.0, dtype=out_dtype, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    fd.extend_paged(q, kp.cuda(), vp.cuda(), table.cuda(), pack_offsets(new).cuda(),
                    torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert bool((out[sum(new):] == 5).all()) and bool((lse[sum(new):] == 5).all())
    at = 0
    for b, n in enumerate(new):
        ref = attend(q[at:at + n], ks[b].cuda(), vs[b].cuda())
        check(out[at:at + n], lse[at:at + n], ref, DT[dtype], lens[b], f"sequence {b} ({n} of {lens[b]})")
        at += n


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 192, 256, 512])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_page_sizes(page, dtype, d):
    """Pages that end inside a tile, lengths that end inside a page."""
    _run([4, 1, 60, 0, 130], [700, 33, 61, 500, 130], 8, 2, d, page, dtype, seed=page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 1), (28, 4), (24, 2), (33, 1), (128, 1), (200, 1)])
def test_groups(Hq, Hkv):
    _run([3, 17, 1], [300, 17, 129], Hq, Hkv, 128, 32, seed=Hq)


@pytest.mark.parametrize("n", [1, 2, 5, 16, 31, 64, 100, 128, 257])
@pytest.mark.parametrize("ctx", [0, 1, 127, 128, 129, 1000])
def test_new_and_cached_lengths(n, ctx):
    _run([n, n], [ctx + n, ctx + n + 3], 8, 2, 64, 16, seed=n + ctx)


def test_more_new_tokens_than_cached():
    """Rows that see nothing: out 0, lse -inf (a length that the queries exceed, and an empty cache)."""
    _run([10, 200, 3], [4, 100, 0], 4, 2, 128, 64, seed=3)


@pytest.mark.parametrize("B", [1, 3, 150])
def test_few_rows_over_long_caches(B):
    """Split over the keys and joined: many pieces a sequence at B = 1."""
    lens = [20011] if B == 1 else [9000, 1, 13000] if B == 3 else [100 + 7 * i for i in range(B)]
    _run([2] * B, [max(n, 2) for n in lens], 8, 1, 128, 64, seed=B)


def test_single_tokens_match_decode():
    """One new token a sequence is decode."""
    lens, Hq, Hkv, d = [700, 33, 1, 2500], 16, 2, 128
    kp, vp, table, ks, vs = (x.cuda() if torch.is_tensor(x) else x for x in paged_cache(lens, 32, Hkv, d, torch.bfloat16, 5, max_pages=90))
    q = torch.randn(4, Hq, d, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fd.extend_paged(q, kp, vp, table, pack_offsets([1] * 4).cuda(), sl, out_dtype=torch.float32)
    dout, dlse = fd.decode_gqa_paged(q, kp, vp, table, sl, out_dtype=torch.float32)
    for b, n in enumerate(lens):
        ref = attend(q[b:b + 1], ks[b].cuda(), vs[b].cuda())
        check(out[b:b + 1], lse[b:b + 1], ref, torch.bfloat16, n)
        check(dout[b:b + 1], dlse[b:b + 1], ref, torch.bfloat16, n)


def test_mixed_batch():
    """Single tokens, drafted ones, chunks and whole prompts in one call."""
    new = [1] * 20 + [4, 4, 5] + [300, 777, 1]
    lens = [50 * i + 1 for i in range(20)] + [900, 4, 2000] + [300, 3000, 4000]
    _run(new, lens, 7, 1, 64, 48, seed=11)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 4, (1300,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 60, (1300,), generator=g))]
    _run(new, lens, 4, 2, 64, 16, seed=6)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16])
def test_output_types(out_dtype):
    _run([9, 70], [400, 70], 8, 2, 128, 16, "f16", out_dtype=out_dtype)


# ---------------------------------------------------------------- E4M3
def _run8(new, lens, Hq, Hkv, d, page, dtype="bf16", seed=0, out_dtype=torch.float32):
    kp, vp, table, ks, vs = paged_cache(lens, page, Hkv, d, torch.float8_e4m3fn, seed)
    g = torch.Generator().manual_seed(seed + 99)
    B = len(lens)
    k_scale, v_scale = ((torch.rand(B, Hkv, generator=g) + 0.5) for _ in range(2))
    q = torch.randn(sum(new), Hq, d, generator=g).to(DT[dtype]).cuda()
    out, lse = fd.extend_paged_fp8(q, kp.cuda(), vp.cuda(), k_scale.cuda(), v_scale.cuda(), table.cuda(),
                                   pack_offsets(new).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   out_dtype=out_dtype)
    at = 0
    for b, n in enumerate(new):
        k = ks[b].double() * k_scale[b].double()[:, None]
        v = vs[b].double() * v_scale[b].double()[:, None]
        ref = attend(q[at:at + n], k.cuda(), v.cuda())
        check(out[at:at + n], lse[at:at + n], ref, DT[dtype], lens[b], f"sequence {b} ({n} of {lens[b]})")
        at += n


@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_e4m3_pages(page, dtype, d):
    _run8([4, 1, 60, 0, 130], [700, 33, 61, 500, 130], 8, 2, d, page, dtype, seed=page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (28, 4), (130, 1)])
def test_e4m3_groups(Hq, Hkv):
    _run8([3, 17, 1], [300, 17, 129], Hq, Hkv, 128, 32, seed=Hq)


def test_e4m3_long():
    _run8([5, 5, 400], [9000, 3, 2000], 8, 1, 128, 128, seed=3)


def test_e4m3_more_new_tokens_than_cached():
    _run8([10, 3], [4, 0], 4, 2, 64, 64, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_e4m3_every_byte(dtype):
    """All 254 finite bytes as K and V, subnormals among them: their exact values."""
    b = torch.arange(256, dtype=torch.uint8)
    b = torch.cat([b[:127], b[128:255]])
    d, n = 64, 254
    rows = torch.stack([b.roll(i) for i in range(n)])[:, :d].contiguous()
    page = 256
    kp = torch.zeros(1, 1, page, d, dtype=torch.uint8)
    kp[0, 0, :n] = rows
    val = rows.view(torch.float8_e4m3fn).double()[:, None]
    q = (torch.randn(6, 1, d, generator=torch.Generator().manual_seed(0)) / 400).to(DT[dtype]).cuda()
    one = torch.ones(1, 1, device="cuda")
    out, lse = fd.extend_paged_fp8(q, kp.cuda(), kp.cuda(), one, one, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                   pack_offsets([6]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                   out_dtype=torch.float32)
    check(out, lse, attend(q, val.cuda(), val.cuda()), DT[dtype], n)


# ---------------------------------------------------------------- pages, streams, graphs
def test_bad_page_is_reported():
    kp, vp, table, ks, vs = paged_cache([300, 100], 32, 2, 64, torch.bfloat16, 1, fill=0.0)
    table[0, 3] = 10 ** 6
    q = torch.randn(8, 4, 64).to(torch.bfloat16).cuda()
    out, lse = fd.extend_paged(q, kp.cuda(), vp.cuda(), table.cuda(), pack_offsets([4, 4]).cuda(),
                               torch.tensor([300, 100], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    assert fd.device_status() == 7
    check(out[4:], lse[4:], attend(q[4:], ks[1].cuda(), vs[1].cuda()), torch.bfloat16, 100, "the other sequence")


def test_lengths_are_clamped_to_the_table():
    kp, vp, table, ks, vs = paged_cache([64], 32, 2, 64, torch.bfloat16, 2)
    q = torch.randn(3, 4, 64).to(torch.bfloat16).cuda()
    args = (q, kp.cuda(), vp.cuda(), table.cuda(), pack_offsets([3]).cuda())
    a = fd.extend_paged(*args, torch.tensor([64], dtype=torch.int32, device="cuda"))
    b = fd.extend_paged(*args, torch.tensor([10 ** 6], dtype=torch.int32, device="cuda"))
    assert torch.equal(a[0], b[0])
    out, lse = fd.extend_paged(*args, torch.tensor([-5], dtype=torch.int32, device="cuda"))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_no_table_columns():
    q = torch.randn(3, 4, 64).to(torch.bfloat16).cuda()
    kp = torch.zeros(1, 2, 32, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = fd.extend_paged(q, kp, kp, torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                               pack_offsets([3]).cuda(), torch.tensor([9], dtype=torch.int32, device="cuda"))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_same_call_twice_same_bits():
    new, lens = [3, 500, 1], [4000, 900, 7000]
    kp, vp, table, _, _ = (x.cuda() if torch.is_tensor(x) else x for x in paged_cache(lens, 64, 2, 128, torch.bfloat16, 1))
    q = torch.randn(504, 16, 128, device="cuda").to(torch.bfloat16)
    args = (q, kp, vp, table, pack_offsets(new).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    a = fd.extend_paged(*args)
    for _ in range(3):
        b = fd.extend_paged(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_with_new_lengths_and_pages():
    """A captured step replayed after its lengths, table and pages changed;
    the rows behind the batch's last token stay as they were."""
    Hq, Hkv, d, page, width = 8, 2, 128, 32, 40
    kp = torch.zeros(120, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    q = torch.randn(64, Hq, d, device="cuda").to(torch.bfloat16)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    sl = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.zeros(64, Hq, d, device="cuda")
    lse = torch.zeros(64, Hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fd.extend_paged(q, kp, vp, table, cu, sl, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.extend_paged(q, kp, vp, table, cu, sl, out=out, lse=lse)
    for seed, (new, lens) in enumerate([([4, 4, 4], [1200, 5, 300]), ([1, 60, 0], [1, 60, 1000]), ([0, 0, 2], [0, 0, 2])]):
        k1, v1, t1, ks, vs = paged_cache(lens, page, Hkv, d, torch.bfloat16, seed, max_pages=width)
        kp[: k1.shape[0]].copy_(k1)
        vp[: v1.shape[0]].copy_(v1)
        table.copy_(t1)
        cu.copy_(pack_offsets(new))
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(5)
        graph.replay()
        at = 0
        for b, n in enumerate(new):
            check(out[at:at + n], lse[at:at + n], attend(q[at:at + n], ks[b].cuda(), vs[b].cuda()), torch.bfloat16, lens[b])
            at += n
        assert bool((out[at:] == 5).all())


def test_page_pool_past_32_bits():
    """Pages whose elements lie past 2^32 in the pool."""
    Hkv, page, d = 8, 256, 128
    P = (1 << 32) // (Hkv * page * d) + 3
    kp = torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    n = 300
    k, v = (torch.randn(n, Hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    ids = [P - 1, 1]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    for x, pool in ((k, kp), (v, vp)):
        pool[ids[0]] = x[:256].transpose(0, 1)
        pool[ids[1], :, :44] = x[256:].transpose(0, 1)
    q = torch.randn(5, 16, d, device="cuda").to(torch.bfloat16)
    out, lse = fd.extend_paged(q, kp, vp, table, pack_offsets([5]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                               out_dtype=torch.float32)
    check(out, lse, attend(q, k, v), torch.bfloat16, n)


def test_e4m3_many_segments_of_one_subtile():
    """Many short items a CTA next to long ones: an engine without blocks of
    its own runs through segments that the other one works on."""
    g = torch.Generator().manual_seed(5)
    new = torch.randint(1, 40, (300,), generator=g).tolist()
    new[::17] = [200 + i for i in range(len(new[::17]))]
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 700, (300,), generator=g))]
    _run8(new, lens, 8, 2, 64, 32, seed=9)
    _run8(new[:120], lens[:120], 8, 2, 128, 16, "f16", seed=10)


def test_past_the_planning_tables():
    """More sequences, and more tiles, than the plan keeps in shared memory."""
    g = torch.Generator().manual_seed(6)
    new = torch.randint(0, 4, (2500,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 200, (2500,), generator=g))]
    _run(new, lens, 2, 1, 64, 16, seed=11)
    _run([4200], [4300], 128, 1, 64, 64, seed=12)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_items_of_one_block(seed, d, dtype):
    """Few tokens over at most a block of keys, which the engines take by
    turns, between items of several blocks and of two sub-tiles, and some
    without any key."""
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, 9, (400,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 120, (400,), generator=g))]
    for i in range(0, 400, 23):
        new[i], lens[i] = 150 + i, 160 + 2 * i      # two sub-tiles
    for i in range(1, 400, 19):
        lens[i] = 129 + 3 * i                       # several blocks of one sub-tile
    for i in range(2, 400, 31):
        lens[i] = new[i] // 2                       # tokens without keys
    _run(new, lens, 6, 2, d, 16, dtype, seed=seed + 20)
    _run8(new[:200], lens[:200], 6, 2, d, 32, dtype, seed=seed + 30)
