"""References and tolerances of the calls around decode.

Attention is checked element by element against the definition in float64.
With w = softmax(s), the kernel's result differs by
  - the rounding of each weight to the 16-bit type of the product with V:
    eps/2 of that type, of every weight, so at most (eps/2) * sum w |V|;
  - the error of a score: d float32 products summed in some order (tensor
    cores may cut where float32 would round: one step, 2^-23, each), and the
    scaling in base 2, (d + 4) * 2^-23 of scale * sum |q_i k_i|, twice (in
    the weight and in the sum of weights), relative to the weight;
  - the float32 sums over m keys, of the weights and of the weights times V,
    and the merge of partial results: (2 m + 64) * 2^-23 of sum w |V|;
  - the exponential on the special-function unit: 2^-21;
  - the rounding of the result to its own type, eps/2 of it.
The log-sum-exp has the score's error, the sum's, and its own rounding.
"""
from __future__ import annotations

import math

import torch


def half_step(dt: torch.dtype) -> float:
    return torch.finfo(dt).eps / 2


def attend(q, k, v, causal=True, scale=None):
    """One sequence in float64: q [n, Hq, d], k, v [m, Hkv, d].  Returns out,
    lse, sum w |V| and the largest scale * sum |q k| of every row."""
    n, Hq, d = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    q, k, v = (t.double() for t in (q, k, v))
    out, mag = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device), None
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    absv, size = torch.zeros_like(out), torch.zeros_like(lse)
    limit = torch.arange(n, device=q.device) + (m - n) if causal else torch.full((n,), m - 1, device=q.device)
    hide = torch.arange(m, device=q.device)[None, :] > limit[:, None]
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kh.T) * scale
        s = s.masked_fill(hide, -math.inf)
        if m:
            mag = ((q[:, h].abs() @ kh.abs().T) * abs(scale)).masked_fill(hide, 0.0)
            size[:, h] = mag.amax(1)
        see = limit >= 0
        if m and bool(see.any()):
            lse[see, h] = torch.logsumexp(s[see], 1)
            w = torch.exp(s[see] - lse[see, h][:, None])
            out[see, h] = w @ vh
            absv[see, h] = w @ vh.abs()
    return out, lse, absv, size


def check(out, lse, ref, dtype, m, what=""):
    """out, lse of the kernel (weights rounded to dtype) against attend()'s ref."""
    r_out, r_lse, absv, size = (t.to(out.device) for t in ref)
    d = out.shape[-1]
    score = (d + 4) * 2.0 ** -23 * size
    sums = (2 * m + 64) * 2.0 ** -23 + 2.0 ** -21
    tol = absv * (half_step(dtype) + 2 * score[..., None] + sums) + half_step(out.dtype) * r_out.abs() + 1e-30
    err = (out.double() - r_out).abs()
    assert bool(torch.isfinite(out).all()), f"{what}: values that are not finite"
    bad = err > tol
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} outputs off, worst {float((err / tol).max()):.2f} of the "
                                 f"tolerance, first at {bad.nonzero()[0].tolist()}")
    if lse is None:
        return
    fin = torch.isfinite(r_lse)
    assert bool((lse[~fin] == -math.inf).all()), f"{what}: a row that sees nothing has lse -inf"
    lt = 2 * score + sums + 2.0 ** -22 * r_lse.abs()
    err = (lse.double() - r_lse).abs()
    assert bool((err[fin] <= lt[fin]).all()), f"{what}: lse off by {float(err[fin].max()):.3e}"


def pack_offsets(lens):
    return torch.tensor([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int32)


def paged_cache(lens, page_size, Hkv, d, dtype, seed, fill=math.nan, spare=3, max_pages=None):
    """Random K/V rows of sequences of these lengths in shuffled pages of a
    pool whose other rows hold ``fill``.  Returns k_pages, v_pages, table,
    and the lists of the sequences' k and v rows [n, Hkv, d] (float32 draws
    rounded to dtype)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g)
    width = max_pages or max(max(need, default=0), 1)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)   # entries behind a sequence's pages are never read
    kp = torch.full((total, Hkv, page_size, d), fill, dtype=torch.float32)
    vp = torch.full((total, Hkv, page_size, d), fill, dtype=torch.float32)
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        k = torch.randn(n, Hkv, d, generator=g).to(dtype).float()
        v = torch.randn(n, Hkv, d, generator=g).to(dtype).float()
        ks.append(k)
        vs.append(v)
        for j in range(need[b]):
            page = int(order[at])
            at += 1
            table[b, j] = page
            rows = slice(j * page_size, min(n, (j + 1) * page_size))
            cnt = rows.stop - rows.start
            kp[page, :, :cnt] = k[rows].transpose(0, 1)
            vp[page, :, :cnt] = v[rows].transpose(0, 1)
    return kp.to(dtype), vp.to(dtype), table, ks, vs


def resize_ref(seqlens, target, table, free, count, page, room=None):
    """fd_resize_pages by one stack and plain loops, on lists.  Returns the
    new lengths, the table, the stack and its height, slots, positions, cu."""
    B, width = len(seqlens), (len(table[0]) if table else 0)
    table, free = [list(r) for r in table], list(free)
    pages = lambda n: -(-n // page)   # noqa: E731
    old, want = list(seqlens), [max(t, 0) for t in target]
    back = [table[b][j] for b in range(B) for j in range(pages(min(want[b], old[b])), pages(old[b]))]
    for page_id in reversed(back):
        free[count] = page_id
        count += 1
    top, new, used_p, used_t = count, list(old), 0, 0
    slots, positions, cu = [], [], [0]
    for b in range(B):
        fits = pages(want[b]) <= width
        need = max(0, pages(want[b]) - pages(old[b])) if fits else 0
        more = max(0, want[b] - old[b]) if fits else 0
        used_p, used_t = used_p + need, used_t + more
        if fits and (need == 0 or used_p <= top) and (more == 0 or room is None or used_t <= room):
            for j in range(pages(old[b]), pages(old[b]) + need):
                count -= 1
                table[b][j] = free[count]
            new[b] = want[b]
            for pos in range(old[b], want[b]):
                slots.append(table[b][pos // page] * page + pos % page)
                positions.append(pos)
        cu.append(len(slots))
    return new, table, free, count, slots, positions, cu
