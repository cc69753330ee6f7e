"""What the rotation is for: products of turned q and k depend on the distance
of their positions alone.

With u = 2^-24: the table's cosines and sines are off by u / 2 each, a pair
(x, y) of length r is turned with an error of u r from these and 2.01 u (|x c| +
|y s|), at most 2.01 u r, in each element, 2.85 u r together: less than 4 u r.  A
product of two heads is then off by 8.1 u times the sum over the pairs of the
product of their lengths (the elements behind `rot` are as they were), and two
such products differ by twice that."""
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


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,H,d,page,rot,far", [(50, 4, 2, 64, 16, 64, 100), (33, 6, 1, 128, 7, 48, 3000), (9, 2, 2, 256, 64, 256, 100000)])
def test_products_depend_on_the_distance_alone(T, Hq, H, d, page, rot, far, pairs):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(T, h, d, device="cuda", generator=g) for h in (Hq, H, H))
    angle = torch.arange(far + 2000, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / -rot)
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    slots = torch.randperm(T, device="cuda", generator=g).to(torch.int32)
    start = torch.randint(0, 1000, (T,), device="cuda", generator=g, dtype=torch.int32)
    products = []
    for shift in (0, 1, far):
        kp, vp = (torch.zeros(-(-T // page), H, page, d, device="cuda") for _ in range(2))
        out = fd.append_rope_paged(k, v, slots, start + shift, table, kp, vp, q=q, interleaved=pairs)
        at = slots.long()
        turned = kp[at // page, :, at % page]
        assert not torch.equal(turned, k) and torch.equal(vp[at // page, :, at % page], v)
        assert torch.equal(turned[..., rot:], k[..., rot:]) and torch.equal(out[..., rot:], q[..., rot:])
        kh = turned.double().repeat_interleave(Hq // H, 1)
        products.append(torch.einsum("thd,shd->hts", out.double(), kh))

    def lengths(x):
        x = x.double()[..., :rot].unflatten(-1, (rot // 2, 2) if pairs else (2, rot // 2))
        return x.square().sum(-1 if pairs else -2).sqrt()

    size = torch.einsum("thi,shi->hts", lengths(q), lengths(k).repeat_interleave(Hq // H, 1))
    for p in products[1:]:
        assert bool(((p - products[0]).abs() <= 16.2 * 2.0 ** -24 * size).all())
    # and on the distance they do depend: the same q at other positions than its own
    moved = torch.einsum("thd,shd->hts", fd.append_rope_paged(k, v, slots, start + 7, table, kp, vp, q=q, interleaved=pairs).double(), kh)
    assert bool(((moved - products[0]).abs() > 16.2 * 2.0 ** -24 * size).any())
