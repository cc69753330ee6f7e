"""Appends with the position rotation (fd_append_rope_paged, _fp8): bit for bit
against the same float32 operations in PyTorch, and within derived bounds of
the rotation in 64 bits.

The bound: two float32 products and their sum, each off by half a step, are
off by 2 * 2^-24 * (|x cos| + |y sin|) at most (a hair more for the steps of
what is already rounded: 2.01); then the rounding to the type, half a step of
the value.  In E4M3 the quotient adds half a float32 step, and the last
rounding is half an E4M3 step, 2^-4 of the value or 2^-10, the half step of its
smallest values, past which 448 saturates."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _table(n, rot):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / -rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _turn(x, row, rot, pairs, dtype):
    """x [T, H, d] turned, in dtype throughout; and the size |x cos| + |y sin| of each element."""
    x = x.to(dtype)
    c, s = row.to(dtype)[:, None].split(rot // 2, dim=2)
    y, size = x.clone(), torch.zeros_like(x)
    at = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    size[..., at[0]], size[..., at[1]] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, size


def _case(T, Hq, H, d, page, rot, dtype, seed, far=4000):
    """q, k, v as views of one projection, slots (some negative), positions."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn(T, Hq + 2 * H, d, device="cuda", generator=g).to(DT[dtype])
    pages = -(-T // page) + 4
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T].to(torch.int32)
    slots[torch.rand(T, device="cuda", generator=g) < 0.1] = -1
    positions = torch.randint(0, far, (T,), device="cuda", generator=g, dtype=torch.int32)
    return wide[:, :Hq], wide[:, Hq:Hq + H], wide[:, Hq + H:], slots, positions, _table(far, rot), pages


def _place(x, slots, like):
    want, live = like.clone(), slots >= 0
    s = slots[live].long()
    want[s // like.shape[2], :, s % like.shape[2]] = x[live]
    return want


SHAPES = [(1, 1, 1, 64, 16, 16), (1, 8, 2, 128, 16, 128), (37, 6, 3, 64, 48, 32), (200, 64, 8, 128, 16, 64), (301, 5, 1, 256, 64, 160),
          (130, 0, 1, 128, 7, 128), (3, 40, 40, 128, 256, 112), (2500, 7, 1, 64, 1, 64), (1025, 3, 3, 256, 32, 256)]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hq,H,d,page,rot", SHAPES)
def test_rows_turned(T, Hq, H, d, page, rot, dtype, pairs):
    q, k, v, slots, pos, table, P = _case(T, Hq, H, d, page, rot, dtype, seed=T + d + rot)
    kp, vp = (torch.full((P, H, page, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    q_out = torch.full((T, Hq, d), 5.0, dtype=DT[dtype], device="cuda")
    k0, v0 = kp.clone(), vp.clone()
    got = fd.append_rope_paged(k, v, slots, pos, table, kp, vp, q=q if Hq else None, q_out=q_out if Hq else None, interleaved=pairs)
    row = table[pos.long()]
    assert torch.equal(vp, _place(v, slots, v0))
    assert torch.equal(kp, _place(_turn(k, row, rot, pairs, torch.float32)[0].to(DT[dtype]), slots, k0))
    if not Hq:
        assert got is None
        return
    live = (slots >= 0)[:, None, None]
    assert got is q_out and torch.equal(q_out, torch.where(live, _turn(q, row, rot, pairs, torch.float32)[0].to(DT[dtype]), 5.0))
    ref, size = _turn(q, row, rot, pairs, torch.float64)
    turn = 2.01 * 2.0 ** -24 * size
    err = (q_out.double() - ref).abs()
    # The float32 result lies within `turn` of the reference, and rounding it
    # adds half a step of what it is: eps/2 of its value, or half of float16's
    # smallest step (2^-24) below its smallest normal value.  The two errors
    # add up, the second one's lower bound as well.
    step = torch.finfo(DT[dtype]).eps / 2 * (ref.abs() + turn)
    tol = turn + (step.clamp(min=2.0 ** -25) if dtype == "f16" else step)
    assert bool((err <= tol)[live.expand_as(err)].all())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,Hq,H,d,page,rot", [
    ([1], 1, 1, 64, 16, 64), ([0, 5, 0, 60], 64, 8, 128, 16, 128), ([1] * 300, 14, 2, 64, 32, 48), ([700, 1], 3, 3, 256, 64, 256),
    ([0, 0, 33], 40, 40, 128, 48, 32), ([3000, 0], 8, 1, 128, 16, 96)])
def test_e4m3_rows_turned(lens, Hq, H, d, page, rot, dtype, pairs):
    T, B = sum(lens), len(lens)
    q, k, v, slots, pos, table, P = _case(T, Hq, H, d, page, rot, dtype, seed=T + rot)
    g = torch.Generator(device="cuda").manual_seed(5)
    ks, vs = ((torch.rand(B, H, device="cuda", generator=g) + 0.1) / 50 for _ in range(2))   # some values saturate
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((P, H, page, d), 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    got = fd.append_rope_paged_fp8(k, v, ks, vs, cu, slots, pos, table, kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn),
                                   q=q, interleaved=pairs)
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(lens, device="cuda"))
    row, live = table[pos.long()], slots >= 0
    assert torch.equal(got[live], _turn(q, row, rot, pairs, torch.float32)[0].to(DT[dtype])[live])
    turned = _turn(k, row, rot, pairs, torch.float32)[0]
    for x, sc, p in ((turned, ks, kp), (v, vs, vp)):
        byte = (x.float() / sc[b][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(p, _place(byte, slots, torch.full_like(p, 1)))
    ref, size = _turn(k, row, rot, pairs, torch.float64)
    scale = ks.double()[b][:, :, None]
    ref, err = ref / scale, 2.01 * 2.0 ** -24 * size / scale
    err = err + 2.0 ** -24 * (ref.abs() + err)
    s = slots[live].long()
    at = kp.view(torch.float8_e4m3fn).double()[s // page, :, s % page]
    tol = err + ((ref.abs() + err) * 2.0 ** -4).clamp(min=2.0 ** -10)
    want = ref.clamp(-448, 448)
    assert bool(((at - want[live]).abs() <= tol[live]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_q_in_place(dtype):
    q, k, v, slots, pos, table, P = _case(77, 8, 2, 128, 16, 64, dtype, seed=3)
    kp, vp = (torch.zeros(P, 2, 16, 128, dtype=DT[dtype], device="cuda") for _ in range(2))
    before = q.clone()
    assert fd.append_rope_paged(k, v, slots, pos, table, kp, vp, q=q, q_out=q) is q
    want = _turn(before, table[pos.long()], 64, False, torch.float32)[0].to(DT[dtype])
    assert torch.equal(q, torch.where((slots >= 0)[:, None, None], want, before))


def test_values_that_are_not_finite_stay_in_their_pair():
    """NaN and infinities reach their pair and nothing else; elements behind rot and V keep their bits."""
    T, H, d, rot = 9, 2, 128, 64
    q, k, v, slots, pos, table, P = _case(T, 4, H, d, 16, rot, "bf16", seed=11)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    k = k.clone()
    k[2, 1, 5], k[3, 0, 40], k[4, 0, 100], k[5, 1, 127] = math.nan, math.inf, -math.inf, math.nan
    kp, vp = (torch.zeros(P, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fd.append_rope_paged(k, v, slots, pos, table, kp, vp)
    got = kp[slots.long() // 16, :, slots.long() % 16]
    want = _turn(k, table[pos.long()], rot, False, torch.float32)[0].to(torch.bfloat16)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
    off = ~torch.isfinite(got)
    assert off.sum() <= 6 and not bool(off[[0, 1, 6, 7, 8]].any())
    assert torch.equal(got[:, :, rot:].view(torch.int16), k[:, :, rot:].view(torch.int16))


def test_bad_slots_and_positions_are_reported_and_skipped():
    q, k, v, slots, pos, table, P = _case(40, 4, 2, 64, 16, 64, "f16", seed=1, far=100)
    slots = torch.arange(40, device="cuda", dtype=torch.int32)
    kp, vp = (torch.full((P, 2, 16, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    for change, status in ((("slots", 3, P * 16), 7), (("slots", 39, 2 ** 31 - 1), 7), (("pos", 5, 100), 9), (("pos", 6, -1), 9),
                           (("pos", 7, 2 ** 31 - 1), 9), (("pos", 8, -2 ** 31), 9)):
        which, t, value = change
        s, p = slots.clone(), pos.clone()
        (s if which == "slots" else p)[t] = value
        kp.fill_(7.0), vp.fill_(7.0)
        out = torch.full((40, 4, 64), 5.0, dtype=torch.float16, device="cuda")
        fd.append_rope_paged(k, v, s, p, table, kp, vp, q=q, q_out=out)
        assert fd.device_status() == status and fd.device_status() == 0
        ok = torch.arange(40, device="cuda") != t
        keep = torch.where(ok, slots, -1)
        p = torch.where(ok, p, 0)
        turned = _turn(k, table[p.long()], 64, False, torch.float32)[0].half()
        assert torch.equal(kp, _place(turned, keep, torch.full_like(kp, 7.0)))
        assert bool((out[t] == 5.0).all()) and not bool((out[ok] == 5.0).all(-1).any())
    # a token that is skipped anyway is not looked at
    s, p = slots.clone(), pos.clone()
    s[2], p[2] = -1, -5
    fd.append_rope_paged(k, v, s, p, table, kp, vp)
    assert fd.device_status() == 0


def test_rows_outside_the_sequences_stay():
    """E4M3: rows ahead of the first sequence and behind the last are skipped, with empty sequences between."""
    T = 30
    q, k, v, slots, pos, table, P = _case(T, 4, 2, 64, 16, 64, "bf16", seed=2)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    cu = torch.tensor([4, 4, 10, 10, 21, 21], dtype=torch.int32, device="cuda")
    sc = torch.full((5, 2), 0.02, device="cuda")
    kp, vp = (torch.full((P, 2, 16, 64), 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    out = torch.full((T, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    fd.append_rope_paged_fp8(k, v, sc, sc, cu, slots, pos, table, kp, vp, q=q, q_out=out)
    keep = torch.where((slots >= 4) & (slots < 21), slots, -1)
    byte = (v.float() / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(vp, _place(byte, keep, torch.full_like(vp, 1)))
    assert bool((out[:4] == 5.0).all()) and bool((out[21:] == 5.0).all()) and not bool((out[4:21] == 5.0).all(-1).any())


@pytest.mark.parametrize("B", [1, 511, 512, 3000, 300000])
def test_many_sequences(B):
    """The sequence of each token among many, empty ones between: its scale, seen in the bytes."""
    g = torch.Generator(device="cuda").manual_seed(B)
    T = 600
    cut = torch.randint(1, T - 1, (B + 1,), device="cuda", generator=g).sort().values
    cu = cut.to(torch.int32)
    k = torch.ones(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    scale = 2.0 ** -torch.randint(0, 9, (B, 1), device="cuda", generator=g).float()
    pos, table = torch.zeros(T, dtype=torch.int32, device="cuda"), _table(1, 64)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    kp, vp = (torch.zeros(T // 16 + 1, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    fd.append_rope_paged_fp8(k, k, scale, scale, cu, slots, pos, table, kp, vp)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cut, t, right=True) - 1
    inside = (b >= 0) & (b < B)
    want = torch.where(inside, 1.0 / scale[b.clamp(0, B - 1), 0], 0.0)
    for p in (kp, vp):
        got = p.view(torch.float8_e4m3fn).float()[t // 16, 0, t % 16]
        assert torch.equal(got, want[:, None].expand(T, 64))


def test_far_positions_and_large_strides():
    """A table past 2^31 bytes' worth of elements, read at its end; rows a long way apart."""
    rot, far = 256, (1 << 23) + 77     # 2^31 elements and more
    table = torch.zeros(far, rot, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    pos = torch.tensor([far - 1, 0, far - 2, 1 << 23], dtype=torch.int32, device="cuda")
    rows = torch.randn(4, rot, device="cuda", generator=g)
    table[pos.long()] = rows
    wide = torch.empty(4, 1 << 20, 256, device="cuda", dtype=torch.float32)[:, :3]   # rows 2^28 elements apart
    wide.copy_(torch.randn(4, 3, 256, device="cuda", generator=g))
    q, k, v = wide[:, :1], wide[:, 1:2], wide[:, 2:]
    slots = torch.arange(4, device="cuda", dtype=torch.int32)
    kp, vp = (torch.zeros(1, 1, 16, 256, device="cuda") for _ in range(2))
    out = fd.append_rope_paged(k, v, slots, pos, table, kp, vp, q=q)
    assert torch.equal(out, _turn(q, rows, rot, False, torch.float32)[0])
    assert torch.equal(kp[0, 0, :4], _turn(k, rows, rot, False, torch.float32)[0][:, 0]) and torch.equal(vp[0, 0, :4], v[:, 0])


def test_pages_far_into_a_pool():
    """Rows behind 2^31 elements of a pool."""
    P, H, page, d = 2100, 8, 512, 256
    kp, vp = (torch.empty(P, H, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([P * page - 1, (P - 2) * page + 3, 5], dtype=torch.int32, device="cuda")
    q, k, v, _, pos, table, _ = _case(3, 1, H, d, 16, 128, "bf16", seed=8)
    fd.append_rope_paged(k, v, slots, pos, table, kp, vp)
    want = _turn(k, table[pos.long()], 128, False, torch.float32)[0].bfloat16()
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kp[s // page, :, s % page], want[t]) and torch.equal(vp[s // page, :, s % page], v[t])


def test_other_stream_and_graph():
    """On a stream of its own, and captured and replayed with new tokens in the same buffers."""
    q, k, v, slots, pos, table, P = _case(64, 8, 2, 128, 16, 128, "bf16", seed=21)
    kp, vp = (torch.zeros(P, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = fd.append_rope_paged(k, v, slots, pos, table, kp, vp, q=q)
    side = torch.cuda.Stream()
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    side.wait_stream(torch.cuda.current_stream())
    got = fd.append_rope_paged(k, v, slots, pos, table, kp2, vp2, q=q, stream=side)
    side.synchronize()
    live = slots >= 0
    assert torch.equal(got[live], want[live]) and torch.equal(kp, kp2) and torch.equal(vp, vp2)
    out = torch.zeros_like(want)
    fd.append_rope_paged(k, v, slots, pos, table, kp2, vp2, q=q, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.append_rope_paged(k, v, slots, pos, table, kp2, vp2, q=q, q_out=out)
    pos.copy_(torch.randint(0, 4000, (64,), device="cuda", dtype=torch.int32))
    slots.copy_(torch.randperm(64, device="cuda"))
    kp2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    row = table[pos.long()]
    assert torch.equal(out, _turn(q, row, 128, False, torch.float32)[0].bfloat16())
    assert torch.equal(kp2, _place(_turn(k, row, 128, False, torch.float32)[0].bfloat16(), slots, torch.zeros_like(kp2)))


def test_as_the_plain_append_then_attention():
    """With cos 1 and sin 0 the call is append_paged; and q and k turned alike leave their product."""
    T, H, d = 50, 2, 64
    q, k, v, slots, pos, table, P = _case(T, 4, H, d, 16, d, "bf16", seed=4)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    still = torch.cat([torch.ones(4000, d // 2), torch.zeros(4000, d // 2)], 1).cuda()
    pools = [torch.zeros(P, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    out = fd.append_rope_paged(k, v, slots, pos, still, pools[0], pools[1], q=q)
    fd.append_paged(k, v, slots, pools[2], pools[3])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3]) and torch.equal(out, q)
