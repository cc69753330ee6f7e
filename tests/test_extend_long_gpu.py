"""Attention of new tokens where one role of the kernel rightly waits for
long: a plan over millions of sequences, segments of a million blocks.  The
values are chosen so that the results are known without a second computation."""
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
