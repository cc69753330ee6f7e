"""How close fd_beam_select's scores are to the definition in float64, and that
its choice between beams follows from it.

With u = 2^-24, half a float32 step, the logarithm of a row's sum is off by
  - the arguments of the exponentials, (x - m) log2 e: a rounded difference, a
    rounded product and log2 e in float32 (0.225 u), 2.23 u of each term's
    distance below the row's largest, through all changes of the running
    maximum; the distances' mean over the softmax is ln V at most;
  - the exponential on the special-function unit: 2^-22, 4 u;
  - up to 7 changes of the running maximum in a part of 8 reads, an exponential
    and a product each: 35 u;
  - the sums of a lane over the part: 31 additions in a read (rows with NaN or
    +inf; 16 otherwise), 7 over reads: 38 u; across the lanes 5 u;
  - the join of the parts, whose sums carry what rounding cuts off: expf with 2
    steps, 4 u, and a product, u;
  - the logarithm: logf with one step of a value below 0.41, 0.5 u, and the
    rounding of its smaller parts.
That is less than (90 + 2.25 ln V) u: 7e-6 at V = 262144.  The score itself is
rounded to float32: u of it."""
import math

import pytest
import torch

import split_kv_fd_gb300 as fd
from beam_util import candidates

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def bound(V):
    return (90 + 2.25 * math.log(V)) * 2.0 ** -24


def _check(x, scores, num):
    """Scores within the bound, and the choice the definition's wherever its
    neighbours are further apart than twice that.  Returns how many neighbours
    of two beams were."""
    out, parents, tokens, _ = (t.cpu() for t in fd.beam_select(x, scores, num))
    R, W, V = x.shape
    tol, pairs = bound(V), 0
    for r in range(R):
        c = candidates(x[r:r + 1], scores[r:r + 1]).flatten()
        best, at = torch.sort(c, descending=True, stable=True)
        best, at = best[:num + 1].cpu(), at[:num + 1].cpu()
        mine = c[(parents[r].long() * V + tokens[r].long()).to(c.device)].cpu()
        err = (out[r].double() - mine).abs()
        assert bool((err <= tol + 2.0 ** -24 * mine.abs()).all()), f"request {r}: off by {float(err.max()):.2e}"
        across = at[:-1] // V != at[1:] // V
        near = across & (best[:-1] - best[1:] <= 2 * tol)
        pairs += int((across & ~near).sum())
        # a group of candidates that near neighbours join may stand in any order, or fall out at the end
        group = torch.cat([torch.zeros(1, dtype=torch.long), (~near).long().cumsum(0)])
        chosen = [(parents[r] * V + tokens[r]).long()[k].item() for k in range(num)]
        for k in range(num):
            allowed = at[group == group[k]].tolist()
            if not (bool(near[-1]) and group[k] == group[-1]):
                assert chosen[k] in allowed, f"request {r}, place {k}: {chosen[k]} for one of {allowed}"
            else:
                assert float(mine[k]) >= float(best[num]) - 2 * tol
    return pairs


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,W,V,K,std", [
    (1, 4, 2, 8, 3.0), (3, 2, 1023, 5, 3.0), (2, 8, 32000, 16, 3.0), (1, 4, 50021, 8, 3.0), (2, 16, 100003, 32, 3.0),
    (1, 2, 262144, 8, 3.0), (2, 5, 131072, 10, 0.05), (2, 3, 262144, 6, 12.0), (40, 8, 8191, 16, 1.0)])
def test_scores_and_the_choice_between_beams(R, W, V, K, std, dtype):
    g = torch.Generator(device="cuda").manual_seed(R + V)
    x = (torch.randn(R, W, V, device="cuda", generator=g) * std).to(DT[dtype])
    # scores as far apart that beams take turns among the best
    scores = -torch.rand(R, W, device="cuda", generator=g) * min(1.0, std)
    assert _check(x, scores, K) >= R


@pytest.mark.parametrize("far", [(11.10, 11.15), (5.0, 5.03), (13.9, 2.2), (0.7, 9.3)])
@pytest.mark.parametrize("V", [131072, 262144])
def test_two_beams_of_one_peak(V, far):
    """Equal logits below a peak: their exponentials' errors do not average out.
    The beams' best scores differ by twice the bound, either way round."""
    x = torch.empty(1, 2, V, device="cuda")
    for w in range(2):
        x[0, w] = -far[w]
        x[0, w, 77 + w] = 0.0
    ln = [math.log1p((V - 1) * math.exp(float(x[0, w, 0]))) for w in range(2)]
    gap = 2 * bound(V)
    for first in range(2):
        other = 1 - first
        s = torch.zeros(2)
        s[first] = -1.0
        want = -1.0 - ln[first] + ln[other] - gap
        s[other] = want
        while float(s[other]) > want:
            s[other] = torch.nextafter(s[other], torch.tensor(-math.inf))
        out, parents, tokens, _ = fd.beam_select(x, s.view(1, 2).cuda(), 2)
        assert parents.tolist() == [[first, other]] and tokens.tolist() == [[77 + first, 77 + other]]
        for k, w in enumerate((first, other)):
            exact = float(s[w]) - ln[w]
            assert abs(float(out[0, k]) - exact) <= bound(V) + 2.0 ** -24 * abs(exact)


def test_a_row_of_many_parts():
    """2^29 logits: more than 65536 parts of one sum, each of 8052.50, which a
    plain float32 sum rounds the same way 2048 times a lane and leaves 3e-5
    off; the bound is 8.1e-6."""
    V, low = 1 << 29, -0.0196533203125
    x = torch.full((1, 1, V), low, dtype=torch.bfloat16, device="cuda")
    x[:, :, 7::8] = 0.0
    assert float(x[0, 0, 0]) == low
    exact = -math.log(V / 8 * (1 + 7 * math.exp(low)))
    out, parents, tokens, _ = fd.beam_select(x, torch.zeros(1, 1, device="cuda"), 3)
    assert tokens.tolist() == [[7, 15, 23]] and parents.tolist() == [[0, 0, 0]]
    assert abs(float(out[0, 0]) - exact) <= bound(V) + 2.0 ** -24 * abs(exact)
