"""Attention of new tokens over very long caches and very many sequences:
where a role of the kernel rightly waits for long, and where sums are long
enough for the tensor cores' way of adding to show."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def test_millions_of_sequences():
    """One token each: its output is its value, its log-sum-exp its score."""
    B, d = 4_000_000, 64
    q = torch.full((B, 1, d), 0.25, dtype=torch.bfloat16, device="cuda")
    v = torch.randint(-100, 100, (B, 1, d), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    out, lse = fd.prefill(q, q, v, torch.arange(B + 1, dtype=torch.int32, device="cuda"), scale=0.5)
    assert fd.device_status() == 0
    assert torch.equal(out, v)
    # 64 * 0.25 * 0.25 * 0.5 = 2: two roundings on the way to base 2 and back
    assert float((lse - 2).abs().max()) <= 2 * 2.0 ** -22


def test_a_hundred_million_keys():
    """A segment takes 1.4 s.  All scores are 0: lse is the logarithm of the
    number of keys that a token sees.  The sums of weights are whole
    multiples of a block's, 2^14, up to 2^34, so they are exact in float32
    but for the last block and the merge."""
    page, width, Hq, T = 1 << 20, 1 << 7, 128, 304
    m = page * width
    kp = torch.zeros(1, 1, page, 64, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, device="cuda")
    q = torch.ones(T, Hq, 64, dtype=torch.float16, device="cuda")
    cu, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [m]))
    _, lse = fd.extend_paged_fp8(q, kp, kp, one, one, table, cu, n)
    assert fd.device_status() == 0
    want = torch.log(m - T + 1.0 + torch.arange(T, device="cuda", dtype=torch.float64))
    assert float((lse.double() - want[:, None]).abs().max()) <= 4 * 2.0 ** -23 * math.log(m)


LINK = 65536   # keys whose sums lie in one accumulator


def _randn(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def _check_row(out, lse, q, k, v, dtype, what):
    """One token, all heads on one K/V head: k, v [m, d] float64, v positive.
    Weights round to dtype; a product may be cut at 2^-24 of the running sum,
    which is half its last value on average: LINK/2 * 2^-24 over a link.  The
    sums of weights are 2^-24 a step of 128 keys and 17 within one, the links
    and pieces some more."""
    d, m = q.shape[-1], k.shape[0]
    s = (q.double() @ k.T) / math.sqrt(d)
    z = torch.logsumexp(s, 1)
    want = torch.exp(s - z[:, None]) @ v
    size = float(((q.double().abs() @ k.abs().T) / math.sqrt(d)).max())
    score = 2 * (d + 4) * 2.0 ** -23 * size
    sums = (min(m, LINK) / 128 + m / LINK + 200) * 2.0 ** -24 + 2.0 ** -21
    rel = ((out.double() - want) / want).abs()
    tol = half_step(dtype) + min(m, LINK) * 2.0 ** -25 + score + sums
    assert float(rel.max()) <= tol, f"{what}: off by {float(rel.max()):.2e}, {float(rel.max()) / tol:.2f} of the tolerance"
    assert float((lse.double() - z).abs().max()) <= score + sums + 2.0 ** -22 * float(z.abs().max()), what


def _paged(m, d, dtype, seed, page=256):
    """m keys and positive values as pages in order, and as float64 rows."""
    k, v = _randn(seed, m, d), torch.rand(m, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)) + 0.5
    k, v = k.to(dtype), v.to(dtype)
    pages = [x.view(m // page, 1, page, d).contiguous() for x in (k, v)]
    return *pages, torch.arange(m // page, dtype=torch.int32, device="cuda")[None], k.double(), v.double()


@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("T,Hq,lg", [(304, 128, 20),     # two sub-tiles, whole items: chains of 16 links
                                     (17, 128, 22),      # cut pieces that are chains themselves
                                     (1, 64, 23),        # one sub-tile that both engines share, cut
                                     (300, 64, 19)])
def test_values_of_one_sign(T, Hq, lg, dtype, d):
    m = 1 << lg
    kp, vp, table, k, v = _paged(m, d, dtype, seed=lg)
    q = _randn(3, T, Hq, d).to(dtype)
    out, lse = fd.extend_paged(q, kp, vp, table, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                               torch.tensor([m], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    for t in {0, T // 2, T - 1}:
        n = m - T + t + 1
        _check_row(out[t], lse[t], q[t], k[:n], v[:n], dtype, f"token {t}")


@pytest.mark.parametrize("dtype,d", [(torch.float16, 128), (torch.bfloat16, 64)])
@pytest.mark.parametrize("T,Hq,lg", [(304, 128, 19), (1, 64, 23)])
def test_values_of_one_sign_e4m3(T, Hq, lg, dtype, d):
    m = 1 << lg
    kp, vp, table, k, v = _paged(m, d, torch.float8_e4m3fn, seed=lg)
    q = _randn(4, T, Hq, d).to(dtype)
    one = torch.ones(1, 1, device="cuda")
    out, lse = fd.extend_paged_fp8(q, kp, vp, one, one * 0.5, table, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                                   torch.tensor([m], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    for t in {0, T // 2, T - 1}:
        n = m - T + t + 1
        _check_row(out[t], lse[t], q[t], k[:n], v[:n] * 0.5, torch.float16, f"token {t}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_single_tokens_over_shared_pages(dtype, d, fp8):
    """One sub-tile a sequence, whole or cut, in chains that both engines share."""
    B, m, Hq = 153, 1 << 18, 64
    kp, vp, table, k, v = _paged(m, d, torch.float8_e4m3fn if fp8 else dtype, seed=13)
    q = _randn(14, B, Hq, d).to(dtype)
    lens = [m - 37 * b for b in range(B)]
    rest = (table.expand(B, -1).contiguous(), torch.arange(B + 1, dtype=torch.int32, device="cuda"),
            torch.tensor(lens, dtype=torch.int32, device="cuda"))
    one = torch.ones(B, 1, device="cuda")
    if fp8:
        out, lse = fd.extend_paged_fp8(q, kp, vp, one, one, *rest, out_dtype=torch.float32)
    else:
        out, lse = fd.extend_paged(q, kp, vp, *rest, out_dtype=torch.float32)
    for b in (0, 1, 70, 151, 152):
        _check_row(out[b], lse[b], q[b], k[:lens[b]], v[:lens[b]], torch.float16 if fp8 else dtype, f"sequence {b}")


@pytest.mark.parametrize("causal", [True, False])
def test_a_long_prompt(causal):
    """Some tiles are one link and some two, beside a short prompt's."""
    lens, d = [50, 70001], 64
    T = sum(lens)
    q = _randn(5, T, 2, d).to(torch.bfloat16)
    k = _randn(6, T, 1, d).to(torch.bfloat16)
    v = (torch.rand(T, 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)) + 0.5).to(torch.bfloat16)
    cu = torch.tensor([0, 50, T], dtype=torch.int32, device="cuda")
    out, lse = fd.prefill(q, k, v, cu, causal=causal, out_dtype=torch.float32)
    for a, n in ((0, 50), (50, 70001)):
        for t in {0, n // 3, 65535, 65536, 65538, n - 1}:
            if t < n:
                keys = slice(a, a + (t + 1 if causal else n))
                _check_row(out[a + t], lse[a + t], q[a + t], k[keys, 0].double(), v[keys, 0].double(), torch.bfloat16, f"{a} {t}")


def test_links_without_a_key_or_with_one_sum():
    """A sub-tile whose last link holds no block of its own, rows that see
    nothing, and scores whose largest moves from link to link."""
    d, m, T, Hq = 64, 65536 + 128, 4, 64          # tiles of 4 tokens: the second sub-tile sees a block more
    kp, vp, table, k, v = _paged(1 << 17, d, torch.float16, seed=9)
    for n in (m + 1, m + 2, m + 3, m + 4):
        q = _randn(n, T, Hq, d).to(torch.float16)
        out, lse = fd.extend_paged(q, kp, vp, table, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
        for t in range(T):
            _check_row(out[t], lse[t], q[t], k[:n - T + t + 1], v[:n - T + t + 1], torch.float16, f"{n} {t}")
    # ever larger scores, and ever smaller ones: each link outweighs the one before, or adds nothing to it
    n, u = 1 << 18, _randn(1, d)
    k = (u * torch.linspace(-4, 4, n, device="cuda")[:, None]).to(torch.float16)
    v = (torch.rand(n, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) + 0.5).to(torch.float16)
    q = u.expand(400, 2, d).to(torch.float16).contiguous()
    for flip in (False, True):
        ka = k.flip(0).contiguous() if flip else k
        cu, ck = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 400], [0, n]))
        out, lse = fd.prefill(q, ka[:, None], v[:, None], cu, ck, out_dtype=torch.float32)
        for t in (0, 399):
            _check_row(out[t], lse[t], q[t], ka[:n - 399 + t].double(), v[:n - 399 + t].double(), torch.float16, f"{flip} {t}")


def test_long_calls_repeat_bit_for_bit():
    kp, vp, table, k, v = _paged(1 << 19, 64, torch.bfloat16, seed=11)
    q = _randn(12, 40, 64, 64).to(torch.bfloat16)
    args = (q, kp, vp, table, torch.tensor([0, 40], dtype=torch.int32, device="cuda"),
            torch.tensor([1 << 19], dtype=torch.int32, device="cuda"))
    a = fd.extend_paged(*args)
    for _ in range(3):
        b = fd.extend_paged(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
