"""The tolerance of the attention tests (serve_util.check), without a GPU: it
takes the definition with its weights rounded as the kernels round them, and
refuses what is off by a little more than that."""
import math

import pytest
import torch

from serve_util import attend, check, half_step

N, M, HQ, HKV, D = 20, 300, 4, 2, 64


def _inputs(dtype, positive=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(n, h, D, generator=g).to(dtype) for n, h in ((N, HQ), (M, HKV), (M, HKV)))
    return q, k, v.abs() if positive else v


def _rounded(q, k, v, dtype, bits_lost=0):
    """The kernel's result: weights to the row's maximum, rounded to dtype
    (`bits_lost` bits below that) for the product with V, their sum not."""
    out, lse = torch.zeros(N, HQ, D), torch.zeros(N, HQ)
    hide = torch.arange(M)[None, :] > torch.arange(N)[:, None] + (M - N)
    for h in range(HQ):
        s = (q[:, h].double() @ k[:, h // (HQ // HKV)].double().T / math.sqrt(D)).masked_fill(hide, -math.inf)
        w = torch.exp(s - s.amax(1, keepdim=True)).float()
        p = w.to(dtype).float()
        if bits_lost:
            step = torch.exp2(torch.floor(torch.log2(w.clamp(min=1e-30))) - (math.log2(0.5 / half_step(dtype)) - bits_lost))
            p = torch.floor(w / step) * step
        out[:, h] = ((p.double() @ v[:, h // (HQ // HKV)].double()) / w.double().sum(1, keepdim=True)).float()
        lse[:, h] = torch.logsumexp(s, 1).float()
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounded_weights_pass(dtype):
    for positive in (False, True):
        q, k, v = _inputs(dtype, positive)
        check(*_rounded(q, k, v, dtype), attend(q, k, v), dtype, M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_of_fewer_bits_do_not(dtype):
    """Two bits less, cut instead of rounded: some 2 half steps too low on average."""
    q, k, v = _inputs(dtype)
    with pytest.raises(AssertionError, match="outputs off"):
        check(*_rounded(q, k, v, dtype, bits_lost=2), attend(q, k, v), dtype, M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_is_just_beyond_does_not(dtype):
    """One output, one log-sum-exp, one value that is not finite, one row that sees nothing."""
    q, k, v = _inputs(dtype)
    ref = attend(q, k, v)
    out, lse = (t.float() for t in ref[:2])
    check(out, lse, ref, dtype, M)
    absv = float(ref[2][7, 1, 5])
    most = half_step(dtype) + (2 * M + 64) * 2.0 ** -23 + 2.0 ** -21 + 2 * (D + 4) * 2.0 ** -23 * float(ref[3][7, 1]) + 2.0 ** -24
    for factor, refused in ((0.9, False), (1.1, True)):
        off = out.clone()
        off[7, 1, 5] += factor * most * absv
        if refused:
            with pytest.raises(AssertionError, match="1 outputs off"):
                check(off, lse, ref, dtype, M)
        else:
            check(off, lse, ref, dtype, M)
    for bad in (math.nan, math.inf):
        off = out.clone()
        off[0, 0, 0] = bad
        with pytest.raises(AssertionError, match="not finite"):
            check(off, lse, ref, dtype, M)
    off = lse.clone()
    off[3, 2] += 1e-3
    with pytest.raises(AssertionError, match="lse off"):
        check(out, off, ref, dtype, M)
    few = attend(q, k[:5], v[:5])     # the first 15 queries see nothing
    out, lse = (t.float() for t in few[:2])
    check(out, lse, few, dtype, 5)
    lse[0, 0] = 0.0
    with pytest.raises(AssertionError, match="sees nothing"):
        check(out, lse, few, dtype, 5)
