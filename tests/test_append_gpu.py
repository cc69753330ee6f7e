"""New K and V rows into a paged cache (fd_append_paged, _fp8): bit for bit,
and in E4M3 against PyTorch's division and conversion."""
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


def _case(T, H, d, page, dtype, seed, extra_heads=0, pages=None):
    """k, v as views of a wider tensor, distinct slots with some negative."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn(T, 2 * H + extra_heads, d, device="cuda", generator=g).to(DT[dtype])
    k, v = wide[:, extra_heads:extra_heads + H], wide[:, extra_heads + H:]
    pages = pages or -(-T // page) + 4
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T].to(torch.int32)
    slots[torch.rand(T, device="cuda", generator=g) < 0.1] = -1
    return k, v, slots, pages


def _gather(pages, slots):
    ps = pages.shape[2]
    s = slots.long()
    raw = pages.view(torch.uint8) if pages.element_size() == 1 else pages
    return raw[s // ps, :, s % ps]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,d,page,extra", [(1, 1, 64, 16, 0), (1, 8, 128, 16, 4), (37, 3, 64, 48, 0),
                                              (200, 8, 128, 16, 7), (1001, 2, 256, 64, 1), (130, 1, 128, 7, 0),
                                              (3, 40, 128, 256, 0)])
def test_rows_land_and_nothing_else_moves(dtype, T, H, d, page, extra):
    k, v, slots, P = _case(T, H, d, page, dtype, seed=T + d, extra_heads=extra)
    kp, vp = (torch.full((P, H, page, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    fd.append_paged(k, v, slots, kp, vp)
    live = slots >= 0
    for x, p in ((k, kp), (v, vp)):
        want = torch.full_like(p, 7.0)
        s = slots[live].long()
        want[s // page, :, s % page] = x[live]
        assert torch.equal(p, want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,H,d,page", [([1], 1, 64, 16), ([0, 5, 0, 60], 8, 128, 16), ([1] * 300, 2, 64, 32),
                                           ([700, 1], 3, 256, 64), ([0, 0, 33], 40, 128, 48)])
def test_e4m3_rows(dtype, lens, H, d, page):
    T, B = sum(lens), len(lens)
    k, v, slots, P = _case(T, H, d, page, dtype, seed=T, extra_heads=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    ks, vs = ((torch.rand(B, H, device="cuda", generator=g) + 0.1) / 50 for _ in range(2))   # some rows saturate
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((P, H, page, d), 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    fd.append_paged_fp8(k, v, ks, vs, cu, slots, kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn))
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(lens, device="cuda"))
    live = slots >= 0
    for x, sc, p in ((k, ks, kp), (v, vs, vp)):
        q = (x.float() / sc[b][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        want = torch.full_like(p, 1)
        s = slots[live].long()
        want[s // page, :, s % page] = q[live]
        assert torch.equal(p, want)


def test_e4m3_every_value_and_ties():
    """All bf16 values that are not NaN, so every tie and every subnormal of
    E4M3, and NaN stays NaN."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    k = bits.view(-1, 1, 128)
    T = k.shape[0]
    one = torch.ones(1, 1, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(T // 16, 1, 16, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    fd.append_paged_fp8(k, k, one, one, cu, slots, kp, vp)
    got = _gather(kp, slots).view(torch.float8_e4m3fn).float().view(-1)
    x = bits.float()
    nan = torch.isnan(x)
    assert bool(torch.isnan(got[nan]).all())
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, 2.0 ** -127, 2.0 ** -126, 1.1e-38, 2.0 ** 125, 2.0 ** 126, 3e38, math.inf,
                                   math.nan, -0.37, 1 / 448, 0.0123, 7.0])
def test_e4m3_is_the_quotient_rounded(dtype, scale):
    """The byte of x / scale for any scale, over all exponents of x."""
    g = torch.Generator().manual_seed(8)
    k = torch.randint(-2 ** 31, 2 ** 31, (512, 4, 64), generator=g).to(torch.int32).view(torch.float32)
    k[256:] = torch.randn(256, 4, 64, generator=g) * 100 * (abs(scale) if 0 < abs(scale) < 1e30 else 1.0)
    k = k.to(DT[dtype])
    want = (k.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    sc = torch.full((1, 4), scale, device="cuda")
    kp, vp = (torch.zeros(512 // 16, 4, 16, 64, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    fd.append_paged_fp8(k.cuda(), k.cuda(), sc, sc, torch.tensor([0, 512], dtype=torch.int32, device="cuda"), slots, kp, vp)
    for pool in (kp, vp):
        got = _gather(pool, slots).view(torch.float8_e4m3fn).float().cpu()
        nan = torch.isnan(want)
        assert bool(torch.isnan(got[nan]).all())
        assert torch.equal(got[~nan], want[~nan]) and torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))


@pytest.mark.parametrize("H,d", [(1, 64), (3, 64), (5, 128), (9, 128), (40, 256)])
@pytest.mark.parametrize("T", [1, 77, 2100, 9000])
def test_tokens_side_by_side(H, d, T):
    """Few heads share a CTA between tokens, many take several rounds."""
    g = torch.Generator(device="cuda").manual_seed(H)
    k, v = (torch.randn(T, H, d, device="cuda", generator=g) for _ in range(2))
    P = -(-T // 16)
    slots = torch.randperm(P * 16, device="cuda", generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    on = slots >= 0
    lens = [T // 2, 0, T - T // 2 - T // 3, T // 3]
    sc = [torch.rand(4, H, device="cuda", generator=g) * 0.01 + 0.005 for _ in range(2)]
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16, torch.float8_e4m3fn):
        src = [x.to(torch.bfloat16) if dt == torch.float8_e4m3fn else x.to(dt) for x in (k, v)]
        pools = [torch.zeros(P, H, 16, d, dtype=torch.uint8 if dt == torch.float8_e4m3fn else dt, device="cuda") for _ in range(2)]
        if dt == torch.float8_e4m3fn:
            fd.append_paged_fp8(*src, *sc, cu, slots, *pools)
            row = torch.repeat_interleave(torch.arange(4, device="cuda"), torch.tensor(lens, device="cuda"))
            src = [(x.float() / s[row][:, :, None]).clamp(-448, 448).to(dt).view(torch.uint8) for x, s in zip(src, sc)]
        else:
            fd.append_paged(*src, slots, *pools)
        for x, pool in zip(src, pools):
            assert torch.equal(_gather(pool, slots[on]), x[on])
            pool.view(P, H, 16, d)[slots[on].long() // 16, :, slots[on].long() % 16] = 0
            assert not bool(pool.view(torch.uint8).any())


def test_rows_outside_the_sequences_are_skipped():
    """E4M3: rows before cu[0] and behind cu[B] belong to nobody."""
    k = torch.randn(10, 2, 64, device="cuda").to(torch.bfloat16)
    slots = torch.arange(10, dtype=torch.int32, device="cuda")
    sc = torch.ones(2, 2, device="cuda")
    cu = torch.tensor([1, 4, 8], dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((1, 2, 16, 64), 3, dtype=torch.uint8, device="cuda") for _ in range(2))
    fd.append_paged_fp8(k, k, sc, sc, cu, slots, kp, vp)
    moved = (kp != 3).any(dim=(0, 1, 3)).tolist()
    assert moved == [False] + [True] * 7 + [False] * 8


def test_slot_past_the_pool_is_reported():
    k = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
    kp, vp = (torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 32, 31], dtype=torch.int32, device="cuda")
    fd.append_paged(k, k, slots, kp, vp)
    assert fd.device_status() == 7
    assert torch.equal(kp[0, :, 0], k[0]) and torch.equal(kp[1, :, 15], k[2])


def test_pool_past_32_bits():
    """A pool of over 2^32 elements: rows land at its end (one page of it is written)."""
    H, page, d = 8, 256, 128
    P = (1 << 32) // (H * page * d) + 2
    kp = torch.empty(P, H, page, d, dtype=torch.bfloat16, device="cuda")
    kp[-1].zero_()
    kp[0].zero_()
    k = torch.randn(4, H, d, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([(P - 1) * page + i for i in (0, 5, 255)] + [3], dtype=torch.int32, device="cuda")
    fd.append_paged(k, k, slots, kp, kp)
    assert torch.equal(kp[-1][:, [0, 5, 255]], k[:3].transpose(0, 1))
    assert torch.equal(kp[0][:, 3], k[3]) and int((kp[0] != 0).any(dim=2).sum()) == H


def test_other_stream():
    k, v, slots, P = _case(500, 4, 128, 16, "bf16", seed=1)
    kp, vp, ka, va = (torch.zeros(P, 4, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    fd.append_paged(k, v, slots, kp, vp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fd.append_paged(k, v, slots, ka, va, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(kp, ka) and torch.equal(vp, va) and math.isfinite(float(kp.float().sum()))
