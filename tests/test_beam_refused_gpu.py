"""A beam search that runs out of pages: a request that is not granted keeps
its scores, flags and logits, appends nothing and chooses again, as the step in
the README does it; requests end through the reordering.  The cache holds each
token's number, so that what a beam reads through its table is its history."""
import random

import pytest
import torch

import split_kv_fd_gb300 as fd

pytestmark = pytest.mark.gpu

VOCAB = 211


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


@pytest.mark.parametrize("spare", [3, 7, 40])
def test_refused_requests_choose_again(spare):
    R, W, page, width, steps = 4, 4, 64, 2, 30
    B, d = R * W, 64
    rng = random.Random(spare)
    g = torch.Generator(device="cuda").manual_seed(spare)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    model = torch.randn(VOCAB, VOCAB, device="cuda", generator=g) * 2     # logits by the last token
    pool = R + spare
    free, free_count = torch.randperm(pool, device="cuda", generator=g).to(torch.int32), i32([pool])
    table, seqlens = torch.zeros(B, width, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    k_pages, v_pages = (torch.full((pool, 1, page, d), -1.0, device="cuda") for _ in range(2))

    def grow(target, tokens):
        """Lengths to their targets; row i of ``tokens`` to the i-th new place."""
        slots = torch.empty(B * page, dtype=torch.int32, device="cuda")
        fd.resize_pages(seqlens, target.to(torch.int32), table, free, free_count, page, slots=slots)
        assert torch.equal(seqlens, target.to(torch.int32))
        n = tokens.numel()
        assert int((slots >= 0).sum()) == n
        rows = tokens.float()[:, None, None].expand(n, 1, d).contiguous()
        fd.append_paged(rows, rows, slots[:n], k_pages, v_pages)

    prompts = [[rng.randrange(VOCAB) for _ in range(rng.randint(3, 25))] for _ in range(R)]
    grow(i32([len(prompts[r]) if w == 0 else 0 for r in range(R) for w in range(W)]),
         torch.tensor([t for p in prompts for t in p], device="cuda"))
    logits = torch.stack([model[p[-1]] for p in prompts])[:, None].repeat(1, W, 1)
    scores = torch.full((R, W), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(R, W, dtype=torch.bool, device="cuda")
    beams = [[list(p)] + [[] for _ in range(W - 1)] for p in prompts]
    made, ended, refused = [0] * R, [False] * R, 0
    for _ in range(steps):
        before = scores.clone(), seqlens.clone(), table.clone()
        new, parents, tokens, over = fd.beam_select(logits, scores, finished=done, eos=7)
        for r in range(R):       # a request ends at its length: its pages come back
            if made[r] == 5 + r and not ended[r]:
                ended[r] = True
        parents[torch.tensor(ended, device="cuda")] = -1
        copies, granted = fd.reorder_pages(parents, seqlens, table, free, free_count, page)
        fd.copy_pages(copies, k_pages, v_pages)
        over[torch.tensor(ended, device="cuda")] = True
        go = granted[:, None] != 0
        scores, done = torch.where(go, new, scores), torch.where(go, over, done)
        goes = (go & ~done).flatten()
        given = granted.tolist()
        for r in range(R):
            rows = slice(r * W, (r + 1) * W)
            if not given[r]:     # whole, as it was
                refused += 1
                assert torch.equal(seqlens[rows], before[1][rows]) and torch.equal(table[rows], before[2][rows])
                assert torch.equal(scores[r], before[0][r])
        grow(seqlens + goes, tokens.flatten()[goes])
        logits = torch.where(go[..., None], model[tokens.clamp(min=0).long()], logits)
        par, tok, gone = parents.tolist(), tokens.tolist(), goes.view(R, W).tolist()
        for r in range(R):
            if given[r]:
                made[r] += not ended[r]
                beams[r] = [beams[r][p] + ([t] if go_on else []) if p >= 0 else [] for p, t, go_on in zip(par[r], tok[r], gone[r])]
        # what each beam reads is its history; each page is one request's or free
        named = []
        for b in range(B):
            own = beams[b // W][b % W]
            at = torch.arange(len(own), device="cuda")
            for pages in (k_pages, v_pages):
                assert pages[table[b, at // page].long(), 0, at % page, 0].long().tolist() == own
            named.append(set(table[b, : -(-len(own) // page)].tolist()))
        whole = [set().union(*named[r * W:(r + 1) * W]) for r in range(R)]
        stack = free[: int(free_count)].tolist()
        assert sum(map(len, whole)) + len(stack) == len(set(stack).union(*whole)) == pool
    assert all(ended) and int(free_count) == pool and (refused > 0) == (spare < 12)
