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


def reorder_ref(parents, lens, table, free, count, page, num_pages=None):
    """fd_reorder_pages by plain loops, on lists.  parents [R][W], lens and
    table by sequence.  Returns lens, table, free, count, copies, granted."""
    R, W = len(parents), len(parents[0])
    lens, table, free = list(lens), [list(t) for t in table], list(free)
    pages = lambda n: -(-n // page)   # noqa: E731
    plans = []
    for r in range(R):
        rows = range(r * W, (r + 1) * W)
        new = [(table[r * W + q][: pages(lens[r * W + q])], lens[r * W + q]) if 0 <= q < W else ([], 0) for q in parents[r]]
        width = max((pages(lens[b]) for b in rows), default=0)
        freed = []
        for j in range(width):
            named = {t[j] for t, _ in new if j < len(t)}
            for b in rows:
                if j < pages(lens[b]) and table[b][j] not in named:
                    named.add(table[b][j])
                    freed.append(table[b][j])
        copies = []   # (beam, place, rows)
        for w, (t, n) in enumerate(new):
            if n % page:
                j = n // page
                for v, (u, m) in enumerate(new):
                    if v != w and j < len(u) and u[j] == t[j] and (m // page > j or v < w):
                        copies.append((w, j, n % page))
                        break
        plans.append((new, freed, copies))
    short = [max(0, len(c) - len(f)) for _, f, c in plans]
    left = count + sum(max(0, len(f) - len(c)) for _, f, c in plans)
    granted, used = [], 0
    for s in short:
        used += s
        granted.append(int(s == 0 or used <= left))
    back = [p for (_, f, _), g in zip(plans, granted) if g for p in f]
    for p in reversed(back):
        free[count] = p
        count += 1
    out = [[-1, -1, 0] for _ in range(R * W)]
    for r, (new, _, copies) in enumerate(plans):
        if not granted[r]:
            continue
        for w, (t, n) in enumerate(new):
            table[r * W + w][: len(t)] = t
            lens[r * W + w] = n
        for w, j, n in copies:
            count -= 1
            out[r * W + w] = [table[r * W + w][j], free[count], n]
            table[r * W + w][j] = free[count]
    return lens, table, free, count, out, granted


class BeamPool:
    """A pool of pages, and requests whose beams grew by steps of choosing and
    writing: a state as a search leaves it, on lists."""

    def __init__(self, rng, R, W, page, width, prompt, grown, spare, ragged=False):
        self.R, self.W, self.page, self.width = R, W, page, width
        self.table = [[rng.randrange(-9, 99) for _ in range(width)] for _ in range(R * W)]   # what lies behind the lengths
        self.lens = [0] * (R * W)
        cap = width * page
        plan = []
        for r in range(R):
            n = min(cap, rng.randint(*prompt))
            plan.append((n, min(cap - n, rng.randint(*grown))))
        self.pool = sum(-(-n // page) + W * (2 + -(-g // page)) for n, g in plan) + spare + 1
        ids = list(range(self.pool))
        rng.shuffle(ids)
        self.free, self.count = ids, self.pool
        for r, (n, g) in enumerate(plan):
            self._grow(r * W, n)
            self.step([[0] * W if q == r else list(range(W)) for q in range(R)])
            left = g
            while left > 0:
                move = min(left, rng.randint(1, max(1, page // 2)))
                for w in range(W):
                    if not (ragged and rng.random() < 0.2):
                        self._grow(r * W + w, self.lens[r * W + w] + move)
                self.step([[rng.randrange(W) for _ in range(W)] if q == r else list(range(W)) for q in range(R)])
                left -= move
        for _ in range(max(0, self.count - spare)):   # no more are free than asked for
            self.count -= 1
            self.free[self.count] = -1

    def _grow(self, b, n):
        for j in range(-(-self.lens[b] // self.page), -(-n // self.page)):
            self.count -= 1
            self.table[b][j] = self.free[self.count]
        self.lens[b] = n

    def step(self, parents):
        self.lens, self.table, self.free, self.count, _, granted = reorder_ref(parents, self.lens, self.table, self.free, self.count, self.page)
        assert all(granted)

    def tensors(self, device="cuda"):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device=device)   # noqa: E731
        return i(self.lens), i(self.table).view(self.R * self.W, self.width), i(self.free), i([self.count])
