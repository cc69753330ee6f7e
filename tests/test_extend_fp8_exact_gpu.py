"""fd_extend_paged_fp8 at the precision it promises, whatever the queries'
type: weights of float16 (half a step, 2^-11), query rows of bf16 scaled by a
power of two a row.  Query rows of all magnitudes, and scales that are not
positive.

A query element keeps its value down to 2^-22 of its row's largest magnitude
(the scaled row's largest lies in [2^8, 2^9), f16's steps below 2^-14 are
2^-24, and 8 significant bits fit above 2^-17); below 2^-25 of it an element
is off by at most 2^-25, which is 2^-33 of the row's largest.  So a score may
be off by scale * 2^-33 * max|q| * sum|k| beside what serve_util counts.  A
weight below 2^-21 of the row's largest (f16's normal numbers, with the
factor 2^7) is off by at most 2^-32 of that, and so is each product with V.
"""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import attend, check, pack_offsets, paged_cache

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
F16_HALF = 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check8(out, lse, q, k, v, what=""):
    """k, v [m, Hkv, d]: the cache's values times their scales, float64."""
    r_out, r_lse, absv, size = attend(q, k, v)
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    scale = 1 / math.sqrt(d)
    if q.dtype == torch.bfloat16 and m:
        top = q.double().abs().amax(-1)                                    # [n, Hq]
        ksum = k.abs().sum(-1).amax(0).repeat_interleave(Hq // Hkv)       # [Hq]
        extra = scale * 2.0 ** -33 * top * ksum
    else:
        extra = torch.zeros_like(size)
    vmax = v.abs().amax((0, 2)).repeat_interleave(Hq // Hkv) if m else torch.zeros(Hq, device=q.device)
    score = (d + 4) * 2.0 ** -23 * size + extra
    sums = (2 * m + 64) * 2.0 ** -23 + 2.0 ** -21
    tol = (absv * (F16_HALF + 2 * score[..., None] + sums) + m * 2.0 ** -32 * vmax[:, None] + 2.0 ** -24 * r_out.abs() + 1e-30)
    assert bool(torch.isfinite(out).all()), f"{what}: values that are not finite"
    err = (out.double() - r_out).abs()
    bad = err > tol
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} outputs off, worst {float((err / tol).max()):.2f} of the "
                                 f"tolerance, first at {bad.nonzero()[0].tolist()}")
    fin = torch.isfinite(r_lse)
    assert bool((lse[~fin] == -math.inf).all()), f"{what}: a row that sees nothing has lse -inf"
    err = (lse.double() - r_lse).abs()
    lt = 2 * score + sums + 2.0 ** -22 * r_lse.abs()
    assert bool((err[fin] <= lt[fin]).all()), f"{what}: lse off by {float(err[fin].max()):.3e}"


def _run(new, lens, Hq, Hkv, d, page, dtype="bf16", seed=0, q=None, k_scale=None, v_scale=None):
    kp, vp, table, ks, vs = paged_cache(lens, page, Hkv, d, torch.float8_e4m3fn, seed)
    g = torch.Generator().manual_seed(seed + 99)
    B = len(lens)
    k_scale, v_scale = ((torch.rand(B, Hkv, generator=g) + 0.5) if s is None else s for s in (k_scale, v_scale))
    if q is None:
        q = torch.randn(sum(new), Hq, d, generator=g)
    q = q.to(DT[dtype]).cuda()
    out, lse = fd.extend_paged_fp8(q, kp.cuda(), vp.cuda(), k_scale.cuda(), v_scale.cuda(), table.cuda(),
                                   pack_offsets(new).cuda(), _i32(lens), out_dtype=torch.float32)
    at = 0
    for b, n in enumerate(new):
        k, v = (x[b].double().cuda() * s[b].double().cuda()[:, None] for x, s in ((ks, k_scale), (vs, v_scale)))
        _check8(out[at:at + n], lse[at:at + n], q[at:at + n], k, v, f"sequence {b} ({n} of {lens[b]})")
        at += n
    return out, lse


@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_pages(page, dtype, d):
    _run([4, 1, 60, 0, 130], [700, 33, 61, 500, 130], 8, 2, d, page, dtype, seed=page)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (28, 4), (130, 1)])
def test_groups(Hq, Hkv, dtype):
    _run([3, 17, 1, 290], [300, 17, 129, 1000], Hq, Hkv, 128, 32, dtype, seed=Hq)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_and_empty(dtype):
    _run([5, 5, 400, 10, 3], [9000, 5, 2000, 4, 0], 8, 1, 128, 128, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_byte(dtype):
    """All 254 finite bytes as K and V, subnormals among them: their exact values."""
    b = torch.arange(256, dtype=torch.uint8)
    b = torch.cat([b[:127], b[128:255]])
    d, n = 64, 254
    rows = torch.stack([b.roll(i) for i in range(n)])[:, :d].contiguous()
    kp = torch.zeros(1, 1, 256, d, dtype=torch.uint8)
    kp[0, 0, :n] = rows
    val = rows.view(torch.float8_e4m3fn).double()[:, None].cuda()
    q = (torch.randn(6, 1, d, generator=torch.Generator().manual_seed(0)) / 400).to(DT[dtype]).cuda()
    one = torch.ones(1, 1, device="cuda")
    out, lse = fd.extend_paged_fp8(q, kp.cuda(), kp.cuda(), one, one, _i32([[0]]), pack_offsets([6]).cuda(), _i32([n]),
                                   out_dtype=torch.float32)
    _check8(out, lse, q, val, val)


# ---------------------------------------------------------------- bf16 queries of all magnitudes
@pytest.mark.parametrize("exponent", [-120, -100, -60, -30, -15, 15, 17, 40, 100, 120])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_one_magnitude(exponent, d):
    """Rows far outside float16's range, K scales that keep the scores near 1."""
    g = torch.Generator().manual_seed(exponent + 200)
    q = torch.randn(64, 8, d, generator=g) * 2.0 ** exponent
    _run([4, 60], [300, 90], 8, 2, d, 32, q=q, k_scale=torch.full((2, 2), 2.0 ** -exponent), seed=5)


def test_rows_of_different_magnitudes_in_a_tile():
    """Each row of a tile with a power of two of its own, rows of zeros among them."""
    g = torch.Generator().manual_seed(11)
    T, Hq, d = 70, 8, 128
    e = torch.randint(-60, 4, (T, Hq, 1), generator=g).float()
    q = torch.randn(T, Hq, d, generator=g) * torch.exp2(e)
    q[::5, 3] = 0
    q[7] = 0
    _run([4, 66], [500, 200], Hq, 2, d, 64, q=q, seed=6)


def test_rows_whose_elements_span_far():
    """Elements of a row from 1 down to 2^-40 of its largest."""
    g = torch.Generator().manual_seed(12)
    T, Hq, d = 40, 4, 128
    e = torch.randint(-40, 1, (T, Hq, d), generator=g).float()
    big = torch.randint(-90, 90, (T, Hq, 1), generator=g).float()
    q = (torch.rand(T, Hq, d, generator=g) + 1) * torch.exp2(e) * torch.where(torch.rand(T, Hq, d, generator=g) < 0.5, -1.0, 1.0)
    _run([3, 37], [400, 260], Hq, 1, d, 16, q=q, seed=7)
    # the same rows at any magnitude, one at a time, give the same scores
    kp, vp, table, ks, vs = paged_cache([260], 16, 1, d, torch.float8_e4m3fn, 8)
    one = torch.ones(1, 1, device="cuda")
    args = (kp.cuda(), vp.cuda())
    rest = (table.cuda(), pack_offsets([1]).cuda(), _i32([260]))
    for t in range(0, T, 9):
        row = q[t:t + 1, :1].to(torch.bfloat16).cuda()
        s = float(big[t, 0])
        a = fd.extend_paged_fp8(row, *args, one, one, *rest, out_dtype=torch.float32)
        b = fd.extend_paged_fp8((row.float() * 2.0 ** s).to(torch.bfloat16), *args, one * 2.0 ** -s, one, *rest,
                                out_dtype=torch.float32)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_largest_and_smallest_queries():
    """bf16's largest numbers, its smallest normal ones and its subnormals."""
    d = 64
    top = torch.finfo(torch.bfloat16).max
    rows = [top, -top, 2.0 ** 127, 2.0 ** -126, 2.0 ** -127, 2.0 ** -133, 0.0]
    g = torch.Generator().manual_seed(13)
    sign = torch.where(torch.rand(len(rows), 1, d, generator=g) < 0.5, -1.0, 1.0)
    q = torch.tensor(rows)[:, None, None] * sign
    for e in (-124, 124):    # K scales that bring one end's scores near 1; the other end's are 0, or left out
        part = q[:3] if e < 0 else q[3:]
        _run([part.shape[0]], [100], 1, 1, d, 16, q=part, k_scale=torch.full((1, 1), 2.0 ** e), seed=14)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite(bad):
    """Its row is NaN, its neighbours' are those without it."""
    kp, vp, table, ks, vs = paged_cache([300], 32, 2, 128, torch.float8_e4m3fn, 9)
    q = torch.randn(20, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    one = torch.ones(1, 2, device="cuda")
    args = (kp.cuda(), vp.cuda(), one, one, table.cuda(), pack_offsets([20]).cuda(), _i32([300]))
    want = fd.extend_paged_fp8(q, *args)
    q[4, 3, 17] = bad
    got = fd.extend_paged_fp8(q, *args)
    for w, x in zip(want, got):
        assert bool(torch.isnan(x[4, 3]).all())
        w[4, 3] = x[4, 3] = 0
        assert torch.equal(w, x)


# ---------------------------------------------------------------- scales
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,lens", [([4, 1], [300, 700]), ([300, 40], [900, 140])])
def test_scales_of_any_sign(new, lens, dtype):
    """K scales of 0 (all keys weigh alike) and below it, V scales too."""
    k_scale = torch.tensor([[0.0, -0.7], [-1.3, 0.9]])
    v_scale = torch.tensor([[0.8, 0.0], [-1.1, -0.6]])
    _run(new, lens, 8, 2, 128, 32, dtype, seed=15, k_scale=k_scale, v_scale=v_scale)
    _run(new, lens, 8, 2, 64, 48, dtype, seed=16, k_scale=-k_scale, v_scale=v_scale.flip(0))


def test_a_scale_that_is_nan():
    """It reaches the rows of its sequence and head that see a key, and no other."""
    lens, new = [200, 300, 2], [3, 200, 4]
    kp, vp, table, ks, vs = paged_cache(lens, 32, 2, 128, torch.float8_e4m3fn, 10)
    q = torch.randn(sum(new), 8, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    sc = torch.rand(3, 2, generator=torch.Generator().manual_seed(3)).cuda() + 0.5
    rest = (table.cuda(), pack_offsets(new).cuda(), _i32(lens))
    want = fd.extend_paged_fp8(q, kp.cuda(), vp.cuda(), sc, sc, *rest)
    for which in (0, 1):
        for b, rows in ((1, slice(3, 203)), (2, slice(205, 207))):   # of sequence 2 the last two tokens see keys
            bad = sc.clone()
            bad[b, 1] = math.nan
            got = fd.extend_paged_fp8(q, kp.cuda(), vp.cuda(), *((bad, sc) if which == 0 else (sc, bad)), *rest)
            hit = torch.zeros(want[0].shape[:2], dtype=torch.bool, device="cuda")
            hit[rows, 4:] = True
            assert bool(torch.isnan(got[0][hit]).all())
            if which == 0:
                assert bool(torch.isnan(got[1][hit]).all())
            assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1][~hit], want[1][~hit])
