"""The serving path around the decode kernels, operator by operator: page
bookkeeping, cache append, attention of new tokens over a paged cache, and
attention over packed prompts.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same
ranges, ``prepare(case, seed)`` makes what a serving loop holds before the
call, and ``run(state)`` makes one pass: with ``own`` true through this
framework's calls, else in elementary torch operations in 32 bits.
``exact(case, seed)`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases
def _listed():
    return [
        # a decode step of a large batch: every request takes one more token,
        # and gives it back (the step is retried): latency of the bookkeeping
        dict(name="pages_step", kind="pages", B=256, page=16, ctx=[1, 32768], new=[1, 1], fresh=0.0, scarce=0.0),
        # admission of new requests next to running ones, then preemption
        dict(name="pages_admit", kind="pages", B=64, page=64, ctx=[1, 16384], new=[1, 4096], fresh=0.75, scarce=0.0),
        # the K/V rows of 16K prompt tokens, views of a fused projection
        dict(name="append_prompt", kind="append", B=8, page=64, ctx=[1, 4096], new=[1500, 2600], Hq=64, Hkv=8, d=128,
             dtype="bf16", cache="same"),
        # one decode step into an E4M3 cache
        dict(name="append_step_e4m3", kind="append", B=256, page=16, ctx=[1, 4096], new=[1, 1], Hq=64, Hkv=8, d=128,
             dtype="bf16", cache="e4m3"),
        # four drafted tokens verified for a few short conversations: latency
        dict(name="extend_verify_small", kind="extend", B=4, page=16, ctx=[700, 2048], new=[4, 4], Hq=32, Hkv=8, d=128,
             dtype="bf16", cache="same"),
        # eight drafted tokens verified for a batch of long ones: bandwidth
        dict(name="extend_verify", kind="extend", B=32, page=64, ctx=[4096, 32768], new=[8, 8], Hq=64, Hkv=8, d=128,
             dtype="bf16", cache="same"),
        # the same over an E4M3 cache
        dict(name="extend_verify_e4m3", kind="extend", B=16, page=128, ctx=[4096, 32768], new=[5, 5], Hq=64, Hkv=8,
             d=128, dtype="bf16", cache="e4m3"),
        # chunked prefill: 2048-token chunks of two long prompts
        dict(name="extend_chunk", kind="extend", B=2, page=128, ctx=[16000, 30000], new=[2048, 2048], Hq=64, Hkv=8,
             d=128, dtype="f16", cache="same"),
        # a mixed batch: single tokens and odd chunks, group of 7, head dim 64
        dict(name="extend_mixed", kind="extend", B=24, page=48, ctx=[0, 9000], new=[1, 777], Hq=28, Hkv=4, d=64,
             dtype="bf16", cache="same"),
        # many short prompts
        dict(name="prompt_short", kind="prompt", B=64, new=[1, 256], Hq=32, Hkv=8, d=128, dtype="bf16", causal=True),
        # a packed batch of prompts of very different lengths
        dict(name="prompt_packed", kind="prompt", B=9, new=[300, 8192], Hq=32, Hkv=4, d=128, dtype="f16", causal=True),
        # one long prompt of an odd length
        dict(name="prompt_long", kind="prompt", B=1, new=[16001, 16001], Hq=64, Hkv=8, d=128, dtype="bf16",
             causal=True),
    ]


def listed():
    cases = []
    for c in _listed():
        c["lens"] = 1   # the seed of the requests' lengths
        for k in ("ctx", "new"):   # a case's fields are plain values: a range is two numbers
            if k in c:
                c[k + "_min"], c[k + "_max"] = c.pop(k)
        cases.append(c)
    return cases


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1))))))


def draw(rng):
    top = {"flops": 0.0, "bytes": 0.0}
    for c in listed():
        for k, x in work(c).items():
            top[k] = max(top[k], x)
    while True:
        kind = rng.choice(["pages", "append", "extend", "extend", "prompt", "prompt"])
        c = {"kind": kind, "lens": rng.randrange(1, 1 << 30), "B": _log(rng, 1, 256)}
        if kind == "pages":
            c |= {"page": rng.choice([1, 16, 32, 48, 64, 128, 256]), "ctx_min": 0, "ctx_max": _log(rng, 16, 32768),
                  "new_min": 1, "new_max": _log(rng, 1, 4096), "fresh": rng.choice([0.0, 0.5, 1.0]),
                  "scarce": rng.choice([0.0, 0.0, 0.3])}
        else:
            G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
            c |= {"Hkv": rng.choice([1, 2, 4, 8])}
            c |= {"Hq": min(64, c["Hkv"] * G) // c["Hkv"] * c["Hkv"], "d": rng.choice([64, 128]),
                  "dtype": rng.choice(["bf16", "f16"]), "new_min": 1}
            if kind == "prompt":
                c |= {"new_max": _log(rng, 1, 16384), "causal": rng.random() < 0.8}
            else:
                c |= {"page": rng.choice([16, 32, 48, 64, 128, 256]), "ctx_min": 0, "ctx_max": _log(rng, 16, 32768),
                      "new_max": _log(rng, 1, 2048 if kind == "extend" else 4096), "cache": rng.choice(["same", "same", "e4m3"])}
        w = work(c)
        if all(w[k] <= top[k] for k in top):
            return c


def _lengths(c):
    """(tokens cached, tokens new) of every request of a case."""
    rng = random.Random(c["lens"])
    ctx, new = [], []
    for _ in range(c["B"]):
        fresh = c["kind"] == "prompt" or rng.random() < c.get("fresh", 0.0)
        ctx.append(0 if fresh else _log(rng, c["ctx_min"], c["ctx_max"]))
        if c["kind"] == "pages" and c["fresh"] and not fresh:
            new.append(1)
        else:
            new.append(_log(rng, c["new_min"], c["new_max"]))
    return ctx, new


def _sees(ctx, new, causal=True):
    """How many (query, key) pairs a request has."""
    return new * ctx + (new * (new + 1) // 2 if causal else new * new)


def _ceil(a, b):
    return -(-a // b)


def work(c):
    ctx, new = _lengths(c)
    T, B = sum(new), c["B"]
    if c["kind"] == "pages":
        pages = sum(_ceil(x + n, c["page"]) - _ceil(x, c["page"]) for x, n in zip(ctx, new))
        # lengths and targets in, offsets and lengths out, a slot and a
        # position a token, each new page from the free list to the table;
        # then the way back
        return {"bytes": float(4 * (2 * B + 2 * B + 1 + 2 * T + 2 * pages + 3 * B + 2 * pages)), "flops": 0.0}
    es = 2
    if c["kind"] == "append":
        one = 1 if c["cache"] == "e4m3" else es
        return {"bytes": float(2 * T * c["Hkv"] * c["d"] * (es + one) + 4 * T), "flops": 0.0}
    kes = 1 if c.get("cache") == "e4m3" else es
    rows = sum(x + n for x, n in zip(ctx, new))
    pairs = sum(_sees(x, n, c.get("causal", True)) for x, n in zip(ctx, new))
    return {"bytes": float(2 * T * c["Hq"] * c["d"] * es + 4 * T * c["Hq"] + 2 * rows * c["Hkv"] * c["d"] * kes),
            "flops": 4.0 * c["d"] * c["Hq"] * pairs}


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(new):
    return _i32([0] + torch.tensor(new).cumsum(0).tolist())


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _paged(c, g, lens):
    """A block table over shuffled pages for these lengths, and the pool's size."""
    need = [_ceil(n, c["page"]) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(c["B"], max(max(need), 1), dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    j = torch.arange(table.shape[1], device="cuda")
    idx = (at[:-1, None] + j).clamp(max=total - 1)
    table = torch.where(j < torch.tensor(need, device="cuda")[:, None], order[idx], table)
    return table, total, order[sum(need):]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lengths(c)
    T, B = sum(new), c["B"]
    s = {"case": c, "new": new, "ctx": ctx}
    if c["kind"] == "pages":
        table, used, left = _paged(c, g, ctx)
        want = sum(_ceil(x + n, c["page"]) - _ceil(x, c["page"]) for x, n in zip(ctx, new))
        room = max(_ceil(x + n, c["page"]) for x, n in zip(ctx, new))
        have = int(want * (1.0 - c["scarce"])) + 5
        pool = used + have
        free = torch.cat([left, used + torch.randperm(have, device="cuda", generator=g).to(torch.int32)])
        s["count"] = _i32([free.numel()])
        s["free"] = torch.cat([free, torch.full((pool - free.numel(),), -1, dtype=torch.int32, device="cuda")])
        wide = torch.zeros(B, max(room, table.shape[1]), dtype=torch.int32, device="cuda")
        wide[:, : table.shape[1]] = table
        s["table"] = wide
        s["seqlens"], s["before"], s["after"] = _i32(ctx), _i32(ctx), _i32([x + n for x, n in zip(ctx, new)])
        room = _ceil(T, 256) * 256  # a padded batch, as a captured step has
        s["slots"], s["positions"] = (torch.zeros(room, dtype=torch.int32, device="cuda") for _ in range(2))
        s["offsets"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        return s
    Hq, Hkv, d, dt = c["Hq"], c["Hkv"], c["d"], DT[c["dtype"]]
    s["offsets"] = _offsets(new)
    if c["kind"] in ("append", "prompt"):
        # the rows of a fused projection: q, k and v of a token side by side
        qkv = _randn(g, T, Hq + 2 * Hkv, d).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if c["kind"] == "prompt":
        return s
    lens = [x + n for x, n in zip(ctx, new)]
    table, pool, _ = _paged(c, g, lens)
    if c["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = ((torch.rand(B, Hkv, device="cuda", generator=g) + 0.5) / 64 for _ in range(2))
    if c["kind"] == "append":
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"), output_size=T)
        pos = torch.arange(T, device="cuda") - s["offsets"].long()[b] + torch.tensor(ctx, device="cuda")[b]
        s["slots"] = (table[b, pos // c["page"]].long() * c["page"] + pos % c["page"]).to(torch.int32)
        s["b"] = b
        kind = torch.float8_e4m3fn if c["cache"] == "e4m3" else dt
        for n in ("k_pages", "v_pages"):
            s[n] = torch.zeros(pool, Hkv, c["page"], d, dtype=torch.uint8 if c["cache"] == "e4m3" else dt, device="cuda").view(kind)
        return s
    s["q"], s["table"], s["seqlens"] = _randn(g, T, Hq, d).to(dt), table, _i32(lens)
    for n in ("k_pages", "v_pages"):
        x = _randn(g, pool, Hkv, c["page"], d)
        s[n] = (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn) if c["cache"] == "e4m3" else x.to(dt)
        del x
    return s


# ---------------------------------------------------------------- plain forms
def _resize(s, target):
    """Every request to its target length, in place: pages released and taken, slots and positions of the new tokens."""
    page, table, free, count = s["case"]["page"], s["table"], s["free"], s["count"]
    B, width = table.shape
    room = s["slots"].numel()
    old, new = s["seqlens"].long(), target.long().clamp(min=0)
    po, pn = (old + page - 1) // page, (new + page - 1) // page
    fits = pn <= width
    need = torch.where(fits, (pn - po).clamp(min=0), 0)
    more = torch.where(fits, (new - old).clamp(min=0), 0)
    j = torch.arange(width, device="cuda")
    gone = (j >= pn[:, None]) & (j < po[:, None])
    back = table[gone]
    top = count.long() + back.numel()
    free[(top - 1 - torch.arange(back.numel(), device="cuda"))] = back
    given = fits & ((need == 0) | (need.cumsum(0) <= top)) & ((more == 0) | (more.cumsum(0) <= room))
    new, pn = torch.where(given, new, old), torch.where(given, pn, po)
    take = (j >= po[:, None]) & (j < pn[:, None])
    n = int(take.sum())
    table[take] = free[top - 1 - torch.arange(n, device="cuda")]
    count.copy_(top - n)
    s["seqlens"].copy_(new)
    off = torch.cat([new.new_zeros(1), (new - old).clamp(min=0).cumsum(0)])
    i = torch.arange(room, device="cuda")
    b = torch.searchsorted(off[1:], i, right=True).clamp(max=B - 1)
    pos = old[b] + i - off[b]
    live = i < off[-1]
    slot = table[b, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return torch.where(live, slot, -1).to(torch.int32), torch.where(live, pos, 0).to(torch.int32), off.to(torch.int32)


def _attend(q, k, v, scale, causal):
    """softmax(scale q K^T) V and its log-sum-exp, one request: q [n, Hq, d], k and v [m, Hkv, d], the last rows of both aligned."""
    n, Hq, d = q.shape
    m, Hkv, _ = k.shape
    q = q.float().view(n, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
    x = torch.matmul(q, k.float().permute(1, 2, 0)).mul_(scale).view(Hkv, Hq // Hkv, n, m)
    if causal:
        x.masked_fill_(torch.arange(m, device="cuda") > torch.arange(n, device="cuda")[:, None] + (m - n), -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(Hkv, -1, m), v.float().permute(1, 0, 2)).view(Hkv, Hq // Hkv, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    return o.permute(2, 0, 1, 3).reshape(n, Hq, d), lse.permute(2, 0, 1).reshape(n, Hq)


def _plain_run(s):
    c = s["case"]
    if c["kind"] == "pages":
        slots, positions, offsets = _resize(s, s["after"])
        table, grown = s["table"].clone(), s["seqlens"].clone()
        _resize(s, s["before"])
        return slots, positions, offsets, table, grown, s["seqlens"], s["free"], s["count"]
    if c["kind"] == "append":
        page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
        for n, pages in (("k", s["k_pages"]), ("v", s["v_pages"])):
            if c["cache"] == "e4m3":
                x = s[n].float() / s[n + "_scale"][s["b"]][:, :, None]
                pages.view(torch.uint8)[page, :, off] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                pages[page, :, off] = s[n]
        return s["k_pages"], s["v_pages"]
    scale, at, outs = c["d"] ** -0.5, 0, []
    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        rows = slice(at, at + n)
        at += n
        if c["kind"] == "prompt":
            outs.append(_attend(s["q"][rows], s["k"][rows], s["v"][rows], scale, c["causal"]))
            continue
        ids = s["table"][b, : _ceil(x + n, c["page"])].long()
        kv = [s[p][ids].transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[: x + n] for p in ("k_pages", "v_pages")] if c["cache"] == "same" else [
            (s[p].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * s[f][b][:, None, None]).transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[: x + n]
            for p, f in (("k_pages", "k_scale"), ("v_pages", "v_scale"))]
        outs.append(_attend(s["q"][rows], kv[0], kv[1], scale, True))
    return torch.cat([o for o, _ in outs]).to(s["q"].dtype), torch.cat([x for _, x in outs])


def _own_run(s):
    import split_kv_fd_gb300 as fd
    c = s["case"]
    if c["kind"] == "pages":
        state = (s["table"], s["free"], s["count"])
        fd.resize_pages(s["seqlens"], s["after"], *state, c["page"], slots=s["slots"], positions=s["positions"], cu_new=s["offsets"])
        table, grown = s["table"].clone(), s["seqlens"].clone()
        fd.resize_pages(s["seqlens"], s["before"], *state, c["page"])
        return s["slots"], s["positions"], s["offsets"], table, grown, s["seqlens"], s["free"], s["count"]
    if c["kind"] == "append":
        if c["cache"] == "e4m3":
            fd.append_paged_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["offsets"], s["slots"], s["k_pages"], s["v_pages"])
        else:
            fd.append_paged(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
        return s["k_pages"], s["v_pages"]
    if c["kind"] == "prompt":
        return fd.prefill(s["q"], s["k"], s["v"], s["offsets"], causal=c["causal"])
    if c["cache"] == "e4m3":
        return fd.extend_paged_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["offsets"], s["seqlens"])
    return fd.extend_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["offsets"], s["seqlens"])


def run(s):
    return _own_run(s) if own else _plain_run(s)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, as float64."""
    x = x.clamp(-448.0, 448.0)
    e = torch.frexp(x.abs())[1].sub(1).clamp(min=-6).double()
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    if c["kind"] == "pages":
        return None
    s = prepare(c, seed)
    if c["kind"] == "append":
        got = []
        for n in ("k", "v"):
            pages = s[n + "_pages"]
            P, H, ps, d = pages.shape
            rows = torch.zeros(P * ps, H, d, dtype=torch.float64, device="cuda")
            x = s[n].double()
            if c["cache"] == "e4m3":
                of = torch.bucketize(torch.arange(x.shape[0], device="cuda"), s["offsets"][1:].long(), right=True)
                x = _exact_e4m3(x / s[n + "_scale"].double()[of].unsqueeze(-1))
            rows.index_copy_(0, s["slots"].long(), x)
            got.append(rows.view(P, ps, H, d).transpose(1, 2))
        return tuple(got)
    # a tenth of a second for every 1e11 operations at the FP64 rate
    if 4.0 * c["d"] * c["Hq"] * sum(n * (x + n) for x, n in zip(s["ctx"], s["new"])) > 1.2e13:
        return None
    T, Hq, d = s["q"].shape
    G = Hq // c["Hkv"]
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    first = s["offsets"].tolist()
    for b in range(c["B"]):
        n, m = first[b + 1] - first[b], s["ctx"][b] + s["new"][b]
        for h in range(c["Hkv"]):
            if c["kind"] == "prompt":
                K, V = (s[t][first[b]:first[b + 1], h].double() for t in ("k", "v"))
            else:
                at = torch.arange(m, device="cuda")
                page, row = s["table"][b].long()[at // c["page"]], at % c["page"]
                K, V = ((s[t].view(torch.uint8)[page, h, row].view(s[t].dtype) if c["cache"] == "e4m3" else s[t][page, h, row]).double()
                        for t in ("k_pages", "v_pages"))
                if c["cache"] == "e4m3":
                    K, V = K * s["k_scale"][b, h].double(), V * s["v_scale"][b, h].double()
            block = max(1, (1 << 28) // max(1, m * G))
            for i in range(0, n, block):
                k = min(n, i + block)
                causal = c.get("causal", True)
                see = m - n + k if causal else m
                q = s["q"][first[b] + i:first[b] + k, h * G:(h + 1) * G].double() / math.sqrt(d)
                x = torch.einsum("igd,jd->gij", q, K[:see])
                if causal:
                    limit = torch.arange(m - n + i, m - n + k, device="cuda")
                    x = x.masked_fill(torch.arange(see, device="cuda")[None, :] > limit[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                out[first[b] + i:first[b] + k, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", torch.exp(x - z[..., None]), V[:see])
                lse[first[b] + i:first[b] + k, h * G:(h + 1) * G] = z.T
                del x
    return out, lse
