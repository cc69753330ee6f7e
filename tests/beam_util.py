"""References of the beam search calls.

Selection is checked against the definition in float64.  A score's error is
that of the logarithm of the sum of exponentials, whose relative error is, in
steps of 2^-23: 2 for the exponential on the special-function unit; the mean
over the softmax of (m - x), at most ln V, for the two roundings of its
argument; one for each of the additions that a term goes through (32 in a
lane's vectors, one a segment, 16 across lanes and warps), one and the
exponential's 2 for each change of the running maximum, counted with the
segments; and a few across the parts.  With at most `segs` segments of 512
elements: (2 + ln V + 48 + 4 segs + 16) * 2^-23; then the rounding of the
score, 2^-24 of it.
"""
from __future__ import annotations

import math

import torch

TOP = 3.4028234663852886e38


def candidates(logits, scores, finished=None, eos=-1):
    """float64 [R, W, V]: every continuation's score, -inf where there is none."""
    x = logits.double()
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=TOP)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = (x - m) - (x - m).exp().sum(-1, keepdim=True).log()
    sc = scores.double()[..., None]
    x = x + sc
    if finished is not None:
        is_eos = torch.arange(x.shape[-1], device=x.device) == eos
        x = torch.where(finished[..., None], torch.where(is_eos, sc, -math.inf), x)
    x = torch.where(sc.isfinite(), x, -math.inf)
    return torch.where(x.isnan() | (x < -TOP), -math.inf, x)


def score_tolerance(V):
    return (66 + math.log(max(V, 2)) + 4 * -(-(V + 8) // 512)) * 2.0 ** -23


def check_select(got, logits, scores, num, finished=None, eos=-1):
    """The four outputs against the definition.  Continuations of one beam are
    in their exact order, of several as far as scores are apart."""
    out, parents, tokens, over = (t.cpu() for t in got)
    R, W, V = logits.shape
    c = candidates(logits, scores, finished, eos)
    best, at = torch.sort(c.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :num + 1].cpu(), at[:, :num + 1].cpu()
    tol = score_tolerance(V)
    flat = parents.long() * V + tokens.long()
    done = finished.cpu() if finished is not None else torch.zeros(R, W, dtype=torch.bool)
    c = c.flatten(1).cpu() if c.numel() <= 1 << 22 else c.flatten(1)
    assert out.shape == parents.shape == tokens.shape == over.shape == (R, num)
    same = 0
    for r in range(R):
        n = int((best[r, :num] > -math.inf).sum())
        assert bool((parents[r, n:] == -1).all() and (tokens[r, n:] == -1).all() and (out[r, n:] == -math.inf).all() and over[r, n:].all())
        f = flat[r, :n]
        assert bool(((parents[r, :n] >= 0) & (parents[r, :n] < W) & (tokens[r, :n] >= 0) & (tokens[r, :n] < V)).all())
        assert f.unique().numel() == n
        mine = c[r, f.to(c.device)].cpu()
        err = (out[r, :n].double() - mine).abs()
        assert bool((err <= tol + 2.0 ** -24 * mine.abs()).all()), f"request {r}: scores off by {float(err.max()):.3e}"
        want = [(t == eos) or bool(done[r, p]) for p, t in zip(parents[r, :n].tolist(), tokens[r, :n].tolist())]
        assert over[r, :n].tolist() == want
        assert bool((mine >= best[r, :n] - 2 * tol).all())
        # of each beam exactly its first ones, in order
        for w in range(W):
            of = f[parents[r, :n] == w]
            if of.numel():
                row = c[r, w * V:(w + 1) * V]
                first = torch.sort(row, descending=True, stable=True)[1][: of.numel()].cpu() + w * V
                assert torch.equal(of, first), f"request {r}, beam {w}: {of.tolist()} for {first.tolist()}"
        gaps = best[r, :n] - best[r, 1:n + 1] if best.shape[1] > n else best[r, :n - 1] - best[r, 1:n]
        beam = at[r, :n + 1] // V
        clear = bool(((gaps > 2 * tol) | (beam[:gaps.numel()] == beam[1:gaps.numel() + 1])).all())
        if clear:
            assert torch.equal(f, at[r, :n]), f"request {r}: {f.tolist()} for {at[r, :n].tolist()}"
            same += 1
    return same
