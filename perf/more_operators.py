"""What a serving loop with rotary positions and beam search needs around the
decode kernels: K and V appended to a paged cache with the position rotation
applied on the way (and q rotated beside them), beam search's selection over
beams and vocabulary, and the reordering of the beams' cached states.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same
ranges, ``prepare(case, seed)`` makes what a serving loop holds before the
call, and ``run(state)`` makes one pass: with ``own`` true through this
framework's calls, else in elementary torch operations.  ``exact(case, seed)``
is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
TOP = 3.4028234663852886e38   # the largest finite float32


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one conversation, rotation of half the head in pairs: latency
        dict(name="rope_one", kind="rope", B=1, page=16, ctx_min=500, ctx_max=2048, new_min=1, new_max=1, Hq=32, Hkv=8, d=128, rot=64,
             pairs=True, dtype="f16", cache="same", lens=1),
        # a decode step of a large batch into an E4M3 cache
        dict(name="rope_step_e4m3", kind="rope", B=256, page=16, ctx_min=1, ctx_max=32768, new_min=1, new_max=1, Hq=64, Hkv=8, d=128,
             rot=128, pairs=False, dtype="bf16", cache="e4m3", lens=1),
        # a mixed batch in float32: odd chunks and single tokens, head dim 64, three K/V heads
        dict(name="rope_mixed_f32", kind="rope", B=24, page=48, ctx_min=0, ctx_max=9000, new_min=1, new_max=777, Hq=21, Hkv=3, d=64,
             rot=32, pairs=False, dtype="f32", cache="same", lens=1),
        # the projections of 16K prompt tokens
        dict(name="rope_prompt", kind="rope", B=8, page=64, ctx_min=1, ctx_max=4096, new_min=1500, new_max=2600, Hq=64, Hkv=8, d=128,
             rot=128, pairs=False, dtype="bf16", cache="same", lens=1),
        # one request of four beams: latency of the selection
        dict(name="select_one", kind="select", R=1, W=4, V=32000, K=8, dtype="bf16", pad=0, done=0.0),
        # odd sizes, rows that start anywhere, some beams finished
        dict(name="select_odd", kind="select", R=17, W=5, V=50021, K=5, dtype="f16", pad=2, done=0.2),
        # a batch of requests, logits as a projection in float32 leaves them
        dict(name="select_f32", kind="select", R=32, W=4, V=128000, K=8, dtype="f32", pad=0, done=0.0),
        # many requests with wide beams and a large vocabulary: bandwidth
        dict(name="select_large", kind="select", R=64, W=8, V=131072, K=16, dtype="bf16", pad=0, done=0.1),
        # a step of a few requests with short contexts: latency of the bookkeeping
        dict(name="reorder_small", kind="reorder", R=4, W=4, page=16, ctx_min=100, ctx_max=2048, grown=100, Hkv=8, d=128, dtype="bf16",
             ends=0.0, start=False, lens=1),
        # a step of a batch with long contexts, a few of the requests at their end
        dict(name="reorder_batch", kind="reorder", R=32, W=8, page=64, ctx_min=1024, ctx_max=32768, grown=500, Hkv=8, d=128, dtype="bf16",
             ends=0.1, start=False, lens=1),
        # wide beams, small pages of an E4M3 cache
        dict(name="reorder_wide_e4m3", kind="reorder", R=24, W=16, page=16, ctx_min=1000, ctx_max=20000, grown=700, Hkv=4, d=64,
             dtype="e4m3", ends=0.1, start=False, lens=1),
        # after the prompts: every request's state to all of its beams
        dict(name="reorder_start", kind="reorder", R=64, W=8, page=128, ctx_min=100, ctx_max=8192, grown=0, Hkv=8, d=128, dtype="bf16",
             ends=0.0, start=True, lens=1),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1))))))


def draw(rng):
    top = {}
    for c in listed():
        best = top.setdefault(c["kind"], {"flops": 0.0, "bytes": 0.0, "held": 0.0})
        for k, x in {**work(c), "held": _held(c)}.items():
            best[k] = max(best[k], x)
    while True:
        kind = rng.choice(["rope", "select", "reorder"])
        c = {"kind": kind}
        if kind == "rope":
            Hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
            c |= {"B": _log(rng, 1, 256), "page": rng.choice([1, 7, 16, 48, 64, 128]), "ctx_min": 0, "ctx_max": _log(rng, 16, 32768),
                  "new_min": 1, "new_max": _log(rng, 1, 4096), "Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 5, 7, 8]), "d": d,
                  "rot": rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]), "pairs": rng.random() < 0.4,
                  "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "cache": rng.choice(["same", "same", "e4m3"]),
                  "lens": rng.randrange(1, 1 << 30)}
        elif kind == "select":
            W, V = rng.randint(1, 16), _log(rng, 100, 262144)
            c |= {"R": _log(rng, 1, 128), "W": W, "V": V, "K": rng.choice([W, W, 2 * W]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                  "pad": rng.choice([0, 0, 1, 2, 3, 64]), "done": rng.choice([0.0, 0.0, 0.1, 0.5])}
        else:
            c |= {"R": _log(rng, 1, 128), "W": rng.randint(1, 16), "page": rng.choice([16, 32, 48, 64, 128, 256]), "ctx_min": 1,
                  "ctx_max": _log(rng, 16, 32768), "grown": _log(rng, 1, 1000), "Hkv": rng.choice([1, 2, 4, 8]),
                  "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f16", "f32", "e4m3"]), "ends": rng.choice([0.0, 0.1, 0.5]),
                  "start": rng.random() < 0.2, "lens": rng.randrange(1, 1 << 30)}
        if _held(c) <= top[kind]["held"] and all(x <= top[kind][k] for k, x in work(c).items()):
            return c


def _ceil(a, b):
    return -(-a // b)


def _lengths(c):
    """(tokens cached, tokens new) of every sequence of an append."""
    rng = random.Random(c["lens"])
    ctx, new = [], []
    for _ in range(c["B"]):
        ctx.append(_log(rng, c["ctx_min"], c["ctx_max"]))
        new.append(_log(rng, c["new_min"], c["new_max"]))
    return ctx, new


def _beams(c):
    """The beams' states before a step and the step's choice: lengths and page
    lists of all R * W beams, parents, and how many pages are named."""
    rng = random.Random(c["lens"])
    W, page = c["W"], c["page"]
    lens, rows, parents, used = [], [], [], 0
    for _ in range(c["R"]):
        prompt = _log(rng, c["ctx_min"], c["ctx_max"])
        grown = 0 if c["start"] else rng.randint(1, c["grown"])
        n = prompt + grown
        head = list(range(used, used + _ceil(prompt, page) if c["start"] else used + prompt // page))
        used += len(head)
        lists = [head] + [[]] * (W - 1) if c["start"] else [head] * W
        # a page further every beam that survived writes pages of its own
        for _ in range(_ceil(n, page) - len(head)):
            if len(lists[0]) > len(head):
                lists = [lists[min(W - 1, int(W * rng.random() ** 2))] for _ in range(W)]
            lists = [x + [used + w] for w, x in enumerate(lists)]
            used += W
        rows += lists
        lens += [n] + [0] * (W - 1) if c["start"] else [n] * W
        ends = rng.random() < c["ends"]
        parents.append([-1] * W if ends else [0] * W if c["start"] else [min(W - 1, int(W * rng.random() ** 2)) for _ in range(W)])
    # pages that later choices left without a beam are not in the pool
    names = {p: i for i, p in enumerate(sorted({p for x in rows for p in x}))}
    return lens, [[names[p] for p in x] for x in rows], parents, len(names)


def _new_copies(c, lens, parents):
    """(parent's row, rows to copy) of each beam whose last page is not its alone any more."""
    got = []
    for r, ps in enumerate(parents):
        seen = set()
        for p in ps:
            n = lens[r * c["W"] + p] % c["page"] if p >= 0 else 0
            if n and p in seen:
                got.append((r * c["W"] + p, n))
            seen.add(p)
    return got


def _row_bytes(c):
    return 2 * c["Hkv"] * c["d"] * SIZE[c["dtype"]]


def _held(c):
    """Bytes that a case keeps on the card."""
    if c["kind"] == "reorder":
        # (an upper bound that needs no page lists)
        return float(c["R"] * (c["ctx_max"] + c["W"] * (c["grown"] + 2 * c["page"])) * _row_bytes(c))
    if c["kind"] == "select":
        return float(c["R"] * c["W"] * (c["V"] + c["pad"]) * SIZE[c["dtype"]])
    return float(c["B"] * (c["ctx_max"] + c["new_max"] + c["page"]) * 2 * c["Hkv"] * c["d"] * SIZE[c["dtype"]])


def work(c):
    if c["kind"] == "rope":
        ctx, new = _lengths(c)
        T, es = sum(new), SIZE[c["dtype"]]
        at, rows = -1, 0   # distinct positions: each row of the table is read once
        for x, n in sorted(zip(ctx, new)):
            rows += max(0, x + n - max(x, at))
            at = max(at, x + n)
        one = SIZE["e4m3"] if c["cache"] == "e4m3" else es
        return {"bytes": float(T * c["d"] * (2 * c["Hq"] * es + 2 * c["Hkv"] * (es + one)) + 8 * T + 4 * rows * c["rot"]),
                "flops": 3.0 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["kind"] == "select":
        live = c["R"] * c["W"] * (1.0 - c["done"])   # a finished beam's logits are not needed
        # a difference, an exponential, a sum and a comparison an element
        return {"bytes": float(live * c["V"] * SIZE[c["dtype"]] + 5 * c["R"] * c["W"] + 13 * c["R"] * c["K"]), "flops": 4.0 * live * c["V"]}
    lens, rows, parents, _ = _beams(c)
    entries = sum(len(x) for x in rows)
    moved = sum(sum(a != b for a, b in zip(rows[r * c["W"] + p], rows[r * c["W"] + i] + [-1] * len(rows[r * c["W"] + p])))
                for r, ps in enumerate(parents) for i, p in enumerate(ps) if p >= 0)
    copied = sum(n for _, n in _new_copies(c, lens, parents))
    B = c["R"] * c["W"]
    # tables, lengths and parents in; changed entries, lengths and the list of
    # copies out; the copied rows in and out
    return {"bytes": float(4 * (entries + 2 * B) + 4 * (moved + 4 * B + c["R"]) + 2 * copied * _row_bytes(c)), "flops": 0.0}


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _noise(g, shape, dtype):
    """Values of a cache: normal in 16 or 32 bits, or E4M3."""
    if dtype == "e4m3":
        x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=g)
        return x.mul_(64).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return torch.empty(shape, dtype=DT[dtype], device="cuda").normal_(generator=g)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "select": _prepare_select, "reorder": _prepare_reorder}[c["kind"]](c, g)


def _prepare_rope(c, g):
    ctx, new = _lengths(c)
    T, B, page, d, dt = sum(new), c["B"], c["page"], c["d"], DT[c["dtype"]]
    s = {"case": c}
    # the rows of a fused projection: q, k and v of a token side by side
    qkv = torch.empty(T, c["Hq"] + 2 * c["Hkv"], d, dtype=dt, device="cuda").normal_(generator=g)
    s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
    # the table of the rotation, once for the whole model
    far = max(x + n for x, n in zip(ctx, new))
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / -c["rot"])
    s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    # the new tokens' places: pages in any order
    need = [_ceil(x + n, page) for x, n in zip(ctx, new)]
    pool = sum(need) + 3
    order = torch.randperm(pool, device="cuda", generator=g)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)
    s["offsets"] = _i32([0] + torch.tensor(new).cumsum(0).tolist())
    s["b"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"), output_size=T)
    pos = torch.arange(T, device="cuda") - s["offsets"].long()[s["b"]] + torch.tensor(ctx, device="cuda")[s["b"]]
    s["positions"] = pos.to(torch.int32)
    s["slots"] = (order[first[s["b"]] + pos // page] * page + pos % page).to(torch.int32)
    e4m3 = c["cache"] == "e4m3"
    if e4m3:
        s["k_scale"], s["v_scale"] = ((torch.rand(B, c["Hkv"], device="cuda", generator=g) + 0.5) / 64 for _ in range(2))
    for n in ("k_pages", "v_pages"):
        s[n] = torch.zeros(pool, c["Hkv"], page, d, dtype=torch.uint8 if e4m3 else dt, device="cuda")
        s[n] = s[n].view(torch.float8_e4m3fn) if e4m3 else s[n]
    return s


def _prepare_select(c, g):
    R, W, V = c["R"], c["W"], c["V"]
    # a projection's padded rows; some tokens forbidden, as a user's mask leaves them
    x = torch.empty(R, W, V + c["pad"], dtype=DT[c["dtype"]], device="cuda").normal_(std=3.0, generator=g)
    x[:, :, V // 2::97] = -math.inf
    scores = -torch.rand(R, W, device="cuda", generator=g) * 8 - 2
    s = {"case": c, "logits": x[:, :, :V], "scores": scores, "eos": V // 3}
    # the first request is at its first token: one beam alone
    s["scores"][0, 1:] = -math.inf
    # (so many of them, in any places)
    done = torch.zeros(R * W, dtype=torch.bool, device="cuda")
    done[torch.randperm(R * W, device="cuda", generator=g)[:int(R * W * c["done"])]] = True
    s["finished"] = done.view(R, W)
    return s


def _prepare_reorder(c, g):
    lens, rows, parents, used = _beams(c)
    B, page = c["R"] * c["W"], c["page"]
    # a page for every beam and a few more are free, the ids in any order
    pool = used + B + 5
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    width = max(len(x) for x in rows) + 1
    table = torch.tensor([x + [0] * (width - len(x)) for x in rows], device="cuda")
    live = torch.arange(width, device="cuda") < _i32([len(x) for x in rows])[:, None]
    table = torch.where(live, order[table], 0)
    free = torch.cat([order[used:], order.new_full((used,), -1)])
    # the state lies in one buffer, as it was before the step in another
    s = {"case": c, "start": torch.cat([table.flatten(), _i32(lens), free, _i32([pool - used])]), "parents": _i32(parents)}
    s["live"] = s["start"].clone()
    table, s["seqlens"], s["free"], s["count"] = s["live"].split([B * width, B, pool, 1])
    s["table"] = table.view(B, width)
    s["k_pages"], s["v_pages"] = (_noise(g, (pool, c["Hkv"], page, c["d"]), c["dtype"]) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, pairs):
    """The first 2 * cos.shape[-1] elements of x [T, H, d] turned by their angles, in 32 bits."""
    x, half = x.float(), cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    u, v = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if pairs else (y[..., :half], y[..., half:2 * half])
    u.copy_(a * cos - b * sin)
    v.copy_(b * cos + a * sin)
    return y


def _plain_rope(s):
    c = s["case"]
    cos, sin = s["rope"][s["positions"].long()].chunk(2, dim=1)
    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    for n in ("k", "v"):
        x = _rotate(s["k"], cos, sin, c["pairs"]) if n == "k" else s["v"]
        pages = s[n + "_pages"]
        if c["cache"] == "e4m3":
            x = x.float() / s[n + "_scale"][s["b"]][:, :, None]
            pages.view(torch.uint8)[page, :, at] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pages[page, :, at] = x.to(pages.dtype)
    return _rotate(s["q"], cos, sin, c["pairs"]).to(s["q"].dtype), s["k_pages"], s["v_pages"]


def _plain_select(s):
    c, x = s["case"], s["logits"].double()   # neighbours of the last choice differ in the last bits
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=TOP)
    top = x.amax(-1, keepdim=True).clamp(min=-TOP)
    x -= top
    x -= x.exp().sum(-1, keepdim=True).log()
    scores = s["scores"].double()[..., None]
    x += scores
    eos = torch.arange(c["V"], device="cuda") == s["eos"]
    done = s["finished"][..., None]
    x = torch.where(done, torch.where(eos, scores, -math.inf), x)
    x = torch.where(scores.isfinite() & x.isfinite(), x, -math.inf)
    x, at = torch.sort(x.flatten(1), dim=1, descending=True, stable=True)
    x, at = x[:, :c["K"]], at[:, :c["K"]]
    some = x > -math.inf
    parents, tokens = torch.where(some, at // c["V"], -1), torch.where(some, at % c["V"], -1)
    over = ~some | (tokens == s["eos"]) | s["finished"].gather(1, parents.clamp(min=0))
    return x.float(), parents.to(torch.int32), tokens.to(torch.int32), over


def _plain_reorder(s):
    c = s["case"]
    R, W, page = c["R"], c["W"], c["page"]
    s["live"].copy_(s["start"])
    old, lens = s["table"].view(R, W, -1).clone(), s["seqlens"].view(R, W).clone()
    width = old.shape[-1]
    par = s["parents"].long()
    kept, par = (par >= 0) & (par < W), par.clamp(0, W - 1)
    j = torch.arange(width, device="cuda")
    new_lens = torch.where(kept, lens.gather(1, par), 0)
    new = old.gather(1, par[..., None].expand(-1, -1, width))
    old_live, new_live = j < ((lens + page - 1) // page)[..., None], j < ((new_lens + page - 1) // page)[..., None]
    # pages that no beam names any more, the first beam's name of each
    gone = old_live.clone()
    for w in range(W):
        gone &= ~(new_live[:, w:w + 1] & (new[:, w:w + 1] == old))
        gone[:, w + 1:] &= ~(old_live[:, w:w + 1] & (old[:, w:w + 1] == old[:, w + 1:]))
    # partly filled last pages that several beams name: all but one get their own
    part = new_lens % page
    last = (new_lens // page).clamp(max=width - 1)
    mine = new.gather(2, last[..., None])                                   # [R, W, 1]
    theirs = new.gather(2, last[:, None, :].expand(-1, W, -1)).transpose(1, 2)   # [R, W, W]: entry of beam v where w's last page is
    there = new_live.gather(2, last[:, None, :].expand(-1, W, -1)).transpose(1, 2)
    full = ((last[:, :, None] + 1) * page) <= new_lens[:, None, :]
    before = torch.arange(W, device="cuda")[:, None] > torch.arange(W, device="cuda")
    copy = (part > 0) & (there & (theirs == mine) & (full | before)).any(-1)
    frees, needs = gone.flatten(1).sum(1), copy.sum(1)
    count = s["count"].long()
    short = (needs - frees).clamp(min=0)
    granted = (short == 0) | (short.cumsum(0) <= count + (frees - needs).clamp(min=0).sum())
    copy &= granted[:, None]
    back = old.transpose(1, 2)[(gone & granted[:, None, None]).transpose(1, 2)]   # in order of request, place, beam
    top = count + back.numel()
    s["free"][top - 1 - torch.arange(back.numel(), device="cuda")] = back
    n = int(copy.sum())
    taken = s["free"][top - 1 - torch.arange(n, device="cuda")]
    s["count"].copy_(top - n)
    copies = torch.full((R, W, 3), -1, dtype=torch.int32, device="cuda")
    copies[..., 2] = 0
    copies[copy] = torch.stack([mine[..., 0][copy], taken, part[copy].to(torch.int32)], dim=1)
    table = torch.where(new_live & granted[:, None, None], new, old)
    table.scatter_(2, last[..., None], torch.where(copy, copies[..., 1], table.gather(2, last[..., None])[..., 0])[..., None])
    s["table"].copy_(table.view(R * W, -1))
    s["seqlens"].copy_(torch.where(granted[:, None], new_lens, lens).flatten())
    copies = copies.view(R * W, 3)
    src, dst, rows = copies[copies[:, 0] >= 0].long().unbind(1)
    for n in ("k_pages", "v_pages"):
        x = s[n].view(torch.uint8) if c["dtype"] == "e4m3" else s[n]
        few = torch.arange(page, device="cuda")[:, None] < rows[:, None, None, None]
        x[dst] = torch.where(few, x[src], x[dst])
    return s["live"], copies, granted.to(torch.int32), s["k_pages"], s["v_pages"]


# ---------------------------------------------------------------- the framework's calls
def _own_rope(s):
    import split_kv_fd_gb300 as fd
    more = dict(q=s["q"], interleaved=s["case"]["pairs"])
    if s["case"]["cache"] == "e4m3":
        q = fd.append_rope_paged_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["offsets"], s["slots"], s["positions"], s["rope"],
                                     s["k_pages"], s["v_pages"], **more)
    else:
        q = fd.append_rope_paged(s["k"], s["v"], s["slots"], s["positions"], s["rope"], s["k_pages"], s["v_pages"], **more)
    return q, s["k_pages"], s["v_pages"]


def _own_select(s):
    import split_kv_fd_gb300 as fd
    return fd.beam_select(s["logits"], s["scores"], s["case"]["K"], finished=s["finished"], eos=s["eos"])


def _own_reorder(s):
    import split_kv_fd_gb300 as fd
    s["live"].copy_(s["start"])
    copies, granted = fd.reorder_pages(s["parents"], s["seqlens"], s["table"], s["free"], s["count"], s["case"]["page"])
    fd.copy_pages(copies, s["k_pages"], s["v_pages"])
    return s["live"], copies, granted, s["k_pages"], s["v_pages"]


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"rope": _own_rope, "select": _own_select, "reorder": _own_reorder}[kind](s)
    return {"rope": _plain_rope, "select": _plain_select, "reorder": _plain_reorder}[kind](s)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, as float64."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.frexp(x.abs())[1].sub(1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    if c["kind"] == "reorder":
        return None   # nothing is computed: rows are moved
    s = prepare(c, seed)
    if c["kind"] == "select":
        got = [], [], [], []
        flat = torch.arange(c["W"] * c["V"], device="cuda").view(c["W"], c["V"])
        for r in range(c["R"]):
            p = s["scores"][r].double()[:, None] + torch.log_softmax(s["logits"][r].double(), -1)
            for w in s["finished"][r].nonzero()[:, 0].tolist():
                p[w] = -math.inf
                p[w, s["eos"]] = s["scores"][r, w].double()
            alive = p > -math.inf
            p, at = p[alive], flat[alive]
            # the K-th largest value, then all above it and the first ones that are it
            k = min(c["K"], p.numel())
            edge = p.kthvalue(p.numel() - k + 1).values if k else 0.0
            above = (p > edge).nonzero()[:, 0]
            pick = torch.cat([above, (p == edge).nonzero()[:, 0][: k - above.numel()]])
            pick = sorted(pick.tolist(), key=lambda i: (-float(p[i]), int(at[i])))
            rest = c["K"] - k
            at = at[pick].tolist()
            beams, tokens = [i // c["V"] for i in at], [i % c["V"] for i in at]
            done = [t == s["eos"] or bool(s["finished"][r, b]) for b, t in zip(beams, tokens)]
            for out, x, none in zip(got, (p[pick].tolist(), beams, tokens, done), (-math.inf, -1, -1, True)):
                out.append(x + [none] * rest)
        kinds = (torch.float64, torch.int32, torch.int32, torch.bool)
        return tuple(torch.tensor(x, dtype=t, device="cuda") for x, t in zip(got, kinds))
    # a turn by an angle as a product of complex numbers
    half = c["rot"] // 2
    row = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]

    def turned(x):
        x = x.double()
        z = x[..., :c["rot"]].unflatten(-1, (half, 2) if c["pairs"] else (2, half))
        z = torch.complex(*z.unbind(-1 if c["pairs"] else -2)) * turn
        z = torch.stack([z.real, z.imag], dim=-1 if c["pairs"] else -2).flatten(-2)
        return torch.cat([z, x[..., c["rot"]:]], dim=-1)

    got = [turned(s["q"])]
    for n in ("k", "v"):
        x = turned(s["k"]) if n == "k" else s["v"].double()
        P, H, page, d = s[n + "_pages"].shape
        if c["cache"] == "e4m3":
            of = torch.bucketize(torch.arange(x.shape[0], device="cuda"), s["offsets"][1:].long(), right=True)
            x = _exact_e4m3(x / s[n + "_scale"].double()[of].unsqueeze(-1))
        rows = torch.zeros(P * page, H, d, dtype=torch.float64, device="cuda")
        rows.index_copy_(0, s["slots"].long(), x)
        got.append(rows.view(P, page, H, d).transpose(1, 2))
    return tuple(got)
