"""The beams' states (fd_reorder_pages, fd_copy_pages) against plain loops on
lists: tables, lengths, the stack, copies and grants, number by number."""
import random

import pytest
import torch

import split_kv_fd_gb300 as fd
from beam_util import BeamPool, reorder_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check(s, parents, status=0):
    """One call on the state s against reorder_ref; the state moves on."""
    lens, table, free, count = s.tensors()
    copies, granted = fd.reorder_pages(_i32(parents), lens, table, free, count, s.page)
    assert fd.device_status() == status
    want = reorder_ref(parents, s.lens, s.table, s.free, s.count, s.page)
    got = (lens.tolist(), table.tolist(), free.tolist(), int(count), copies.tolist(), granted.tolist())
    for name, a, b in zip(("lens", "table", "stack", "count", "copies", "granted"), got, want):
        assert a == b, name
    s.lens, s.table, s.free, s.count = want[:4]
    return want[4], want[5]


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("R,W,page,width,prompt,grown", [
    (1, 1, 16, 4, (1, 40), (0, 20)), (1, 4, 16, 20, (5, 100), (1, 60)), (5, 3, 7, 40, (1, 200), (0, 50)), (3, 32, 4, 50, (1, 60), (1, 40)),
    (2, 16, 1, 300, (100, 250), (1, 30)), (9, 8, 64, 9, (1, 300), (0, 200)), (1, 5, 2, 1300, (500, 2400), (10, 200)),
    (40, 2, 48, 6, (0, 100), (0, 100))])
def test_steps(R, W, page, width, prompt, grown, seed):
    rng = random.Random(seed * 100 + W)
    s = BeamPool(rng, R, W, page, width, prompt, grown, spare=R * W, ragged=seed == 2)
    for step in range(4):
        ends = 0.0 if step < 2 else 0.3
        parents = [[-1] * W if rng.random() < ends else [rng.randrange(W) if rng.random() > ends / 2 else -1 for _ in range(W)]
                   for _ in range(R)]
        _, granted = _check(s, parents)
        assert all(granted)


@pytest.mark.parametrize("spare", [0, 1, 3, 7, 20])
def test_too_few_pages(spare):
    """Some requests are refused and stay as they were, whole; others behind them go on."""
    seen = set()
    for seed in range(8):
        rng = random.Random(seed)
        s = BeamPool(rng, 6, 4, 16, 12, (3, 90), (1, 40), spare=spare)
        # every beam from one: three copies a request, as many as come back or more
        parents = []
        for r in range(6):
            w = rng.randrange(4)
            parents.append(rng.choice([[w] * 4, [w, w, -1, -1], [0, 1, 2, 3], [-1] * 4]))
        # lengths of 0 but one: nothing comes back
        for r in rng.sample(range(6), 3):
            for w in range(1, 4):
                s.lens[r * 4 + w] = 0
            parents[r] = [0, 0, 0, 0]
        _, granted = _check(s, parents)
        seen |= set(granted)
        _check(s, [[0, 0, 1, 1]] * 6)
    assert seen == ({0, 1} if spare < 7 else seen)


def test_start_and_end_undo_each_other():
    """Beams start from a prompt and end again: the stack is what it was."""
    rng = random.Random(3)
    s = BeamPool(rng, 5, 6, 16, 10, (1, 150), (0, 0), spare=40)
    for r in range(5):
        for w in range(1, 6):
            s.lens[r * 6 + w] = 0
    before = list(s.free[: s.count]), s.count, list(s.lens)
    copies, granted = _check(s, [[0] * 6] * 5)
    assert sum(c[0] >= 0 for c in copies) == 5 * sum(1 for r in range(5) if s.lens[r * 6] % 16) and all(granted)
    _check(s, [[0] + [-1] * 5] * 5)
    assert (list(s.free[: s.count]), s.count, list(s.lens)) == before


def test_beams_that_already_share_a_partly_filled_page():
    """A table written to all beams by hand: the first keeps the page, and a
    page that one beam has full and another in part is copied for the latter."""
    s = BeamPool(random.Random(1), 2, 4, 16, 6, (20, 20), (0, 0), spare=12)
    for w in range(4):
        s.table[w] = list(s.table[0])
        s.lens[w] = 20
    copies, _ = _check(s, [[0, 1, 2, 3], [0, -1, -1, -1]])
    assert [c[2] for c in copies[:4]] == [0, 4, 4, 4]
    s = BeamPool(random.Random(2), 1, 3, 16, 6, (40, 40), (0, 0), spare=12)
    for w in range(3):
        s.table[w] = list(s.table[0])
    s.lens = [35, 32, 20]      # full, full, 4 rows of the second page
    s.table[1][2] = s.free[s.count - 1]
    s.count -= 1
    copies, _ = _check(s, [[2, 0, 0]])
    assert copies[0] == [s.table[1][1], s.table[0][1], 4] and copies[1][2] == 0 and copies[2][2] == 3


def test_bad_parents_and_pages():
    s = BeamPool(random.Random(5), 2, 3, 16, 8, (30, 60), (5, 20), spare=8)
    state = s.tensors()
    _check(s, [[0, 3, 1], [2 ** 31 - 1, 2, 2]], status=9)        # as if they ended
    _check(s, [[-2 ** 31, 0, -7], [1, 1, 2]])
    del state
    # ids that name no page are moved, not released and not copied
    s = BeamPool(random.Random(6), 1, 2, 16, 4, (20, 20), (0, 0), spare=4)
    lens, table, free, count = s.tensors()
    pool = free.numel()
    for bad in (-1, pool, 2 ** 31 - 1, -2 ** 31):
        t, n, f, c = table.clone(), _i32([20, 20]), free.clone(), count.clone()
        t[0, 1] = bad
        copies, granted = fd.reorder_pages(_i32([[0, 0]]), n, t, f, c, 16)
        assert fd.device_status() == 7 and fd.device_status() == 0
        assert copies.tolist() == [[-1, -1, 0]] * 2 and t[1, 1] == bad and granted.tolist() == [1]
        t[0, 0] = t[0, 1] = bad
        had = int(c)
        fd.reorder_pages(_i32([[-1, -1]]), n, t, f, c, 16)
        assert fd.device_status() == 7 and n.tolist() == [0, 0] and int(c) >= had and bool(((f >= 0) & (f < pool) | (f == -1)).all())
    # a stack that does not hold what it says: the copy has no page, and nothing else is written
    t, n, f, c = table.clone(), _i32([20, 0]), torch.full_like(free, pool + 5), count.clone()
    copies, _ = fd.reorder_pages(_i32([[0, 0]]), n, t, f, c, 16)
    assert fd.device_status() == 7 and copies.tolist() == [[-1, -1, 0]] * 2 and t[1, 1] == -1
    # pages given back twice would pass the stack's end
    t, n, f = table.clone(), _i32([20, 20]), free.clone()
    c = _i32([pool])
    fd.reorder_pages(_i32([[-1, -1]]), n, t, f, c, 16)
    assert fd.device_status() == 7 and int(c) == pool
    # lengths outside the table
    t, n, c = table.clone(), _i32([2 ** 31 - 1, -5]), _i32([0])
    fd.reorder_pages(_i32([[0, -1]]), n, t, free.clone(), c, 16)
    assert n.tolist() == [64, 0]
    fd.device_status()


def test_empty_sizes():
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    copies, granted = fd.reorder_pages(e.view(0, 4), e, e.view(0, 3), e, _i32([0]), 16)
    assert copies.shape == (0, 3) and granted.shape == (0,)
    lens = _i32([0, 0])
    copies, granted = fd.reorder_pages(_i32([[0, 0]]), lens, e.view(2, 0), e, _i32([0]), 16)   # a table of no pages
    assert lens.tolist() == [0, 0] and granted.tolist() == [1]
    fd.copy_pages(torch.zeros(0, 3, dtype=torch.int32, device="cuda"), *(torch.zeros(1, 1, 16, 64, device="cuda") for _ in range(2)))


def test_many_requests():
    """More requests than the sums take in one pass, with refusals among them."""
    R, W, page = 2500, 2, 4
    rng = random.Random(7)
    lens = [rng.randint(1, 11) if w == 0 or rng.random() < 0.5 else 0 for _ in range(R) for w in range(W)]
    ids = list(range(8 * R))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(3)] for _ in range(R * W)]
    s = BeamPool(rng, 1, 1, 4, 1, (1, 1), (0, 0), spare=0)
    s.R, s.W, s.width, s.page, s.lens, s.table = R, W, 3, page, lens, table
    s.free, s.count = ids + [-1] * (8 * R - len(ids)), 700
    parents = [rng.choice([[0, 0], [0, 1], [1, 0], [1, 1], [-1, 0], [-1, -1]]) for _ in range(R)]
    _, granted = _check(s, parents)
    assert 0 < sum(granted)
    s.count = 3
    _, granted = _check(s, [[0, 0]] * R)
    assert all(granted)      # (what others give back is enough)
    # each request starts a second beam, and one in four needs no page for it: after 500 pages the others are refused
    s.lens = [n for r in range(R) for n in (r % 12 + 1, 0)]
    s.count = 500
    _, granted = _check(s, [[0, 0]] * R)
    assert sum(granted) == sum(1 for r in range(R) if (r % 12 + 1) % 4 == 0) + 500


@pytest.mark.parametrize("spare", [3, 700])
def test_wide_tables_of_many_requests(spare):
    """More tiles of tables than are added up in one pass, most of them empty."""
    rng = random.Random(spare)
    s = BeamPool(rng, 220, 2, 2, 1300, (1, 40), (0, 10), spare=spare)
    s.lens[0:2], s.lens[4] = [2599, 2600], 0        # one request over all of its tiles
    for b, n in ((0, 2599), (1, 2600)):
        s.table[b] = [100000 + b * 1300 + j if j >= 5 else s.table[b][j] for j in range(1300)]
    s.free += [-1] * (110000 - s.pool)
    for _ in range(3):
        _check(s, [rng.choice([[0, 0], [1, 1], [0, 1], [1, 0], [-1, 0], [1, -1]]) for _ in range(220)])
    _check(s, [[-1, -1]] * 220)
    assert not any(s.lens)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3", "u8"])
@pytest.mark.parametrize("H,page,d", [(1, 16, 64), (8, 64, 128), (3, 7, 256), (2, 256, 128), (40, 1, 64)])
def test_copies(H, page, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(page)
    P = 40
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8, "u8": torch.uint8}[dtype]
    kp, vp = (torch.randint(0, 255, (P, H, page, d), device="cuda", generator=g).to(dt) for _ in range(2))
    order = torch.randperm(P, device="cuda", generator=g).tolist()
    copies = [[order[i], order[20 + i], int(n)] for i, n in enumerate([1, page, page // 2, 0, page - 1, page + 5, -3])]
    copies += [[-1, -1, 0], [-1, order[30], 5], [order[0], order[31], 1], [order[0], order[32], page]]
    k0, v0 = kp.clone(), vp.clone()
    view = (lambda t: t.view(torch.float8_e4m3fn)) if dtype == "e4m3" else (lambda t: t)   # noqa: E731
    fd.copy_pages(_i32(copies), view(kp), view(vp))
    for f, t, n in copies:
        n = min(n, page)
        if f >= 0 and n > 0:
            k0[t, :, :n], v0[t, :, :n] = k0[f, :, :n].clone(), v0[f, :, :n].clone()
    assert torch.equal(kp, k0) and torch.equal(vp, v0) and fd.device_status() == 0


def test_copies_of_no_page():
    kp, vp = (torch.randn(4, 2, 16, 64, device="cuda") for _ in range(2))
    k0 = kp.clone()
    for bad in ([4, 1, 3], [0, 4, 3], [0, -1, 3], [2 ** 31 - 1, 0, 1], [0, 2 ** 31 - 1, 1]):
        fd.copy_pages(_i32([bad]), kp, vp)
        assert fd.device_status() == 7 and torch.equal(kp, k0)


def test_copies_far_into_a_pool():
    """Pages behind 2^31 elements and 2^32 bytes."""
    P, H, page, d = 2100, 8, 512, 256
    kp = torch.empty(P, H, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty(P, H, page, d, dtype=torch.bfloat16, device="cuda")
    for t in (kp, vp):
        t[[0, 1, P - 2, P - 1]] = torch.randn(4, H, page, d, device="cuda").bfloat16()
    want = kp[0].clone(), vp[P - 1].clone(), kp[1].clone()
    fd.copy_pages(_i32([[0, P - 2, page], [P - 1, 1, 100]]), kp, vp)
    assert torch.equal(kp[P - 2], want[0]) and torch.equal(vp[1, :, :100], want[1][:, :100]) and torch.equal(kp[1, :, 100:], want[2][:, 100:])


def test_stream_workspace_and_graph():
    """A captured step, replayed with other parents, on a workspace of rubbish."""
    rng = random.Random(12)
    s = BeamPool(rng, 3, 4, 16, 12, (10, 90), (5, 60), spare=14)
    lens, table, free, count = s.tensors()
    ws = torch.full((fd.workspace_size_reorder(3, 4, 12),), 0xff, dtype=torch.uint8, device="cuda")
    parents = _i32([[0, 1, 2, 3]] * 3)
    copies, granted = fd.reorder_pages(parents, lens, table, free, count, 16, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.reorder_pages(parents, lens, table, free, count, 16, copies=copies, granted=granted, workspace=ws)
    for _ in range(6):
        step = [[rng.randrange(4) for _ in range(4)] for _ in range(3)]
        parents.copy_(_i32(step))
        graph.replay()
        s.lens, s.table, s.free, s.count, c, g = reorder_ref(step, s.lens, s.table, s.free, s.count, 16)
        assert (lens.tolist(), table.tolist(), free.tolist(), int(count), copies.tolist(), granted.tolist()) == (s.lens, s.table, s.free, s.count, c, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fd.reorder_pages(_i32([[3, 2, 1, 0]] * 3), lens.view(3, 4), table, free, count, 16, stream=side)
    side.synchronize()
    want = reorder_ref([[3, 2, 1, 0]] * 3, s.lens, s.table, s.free, s.count, 16)
    assert (lens.tolist(), table.tolist(), got[0].tolist()) == (want[0], want[1], want[4])


def test_refusals():
    s = BeamPool(random.Random(1), 1, 2, 16, 4, (20, 20), (0, 0), spare=4)
    lens, table, free, count = s.tensors()
    par = _i32([[0, 1]])
    with pytest.raises(ValueError):
        fd.reorder_pages(par.long(), lens, table, free, count, 16)
    with pytest.raises(ValueError):
        fd.reorder_pages(par, lens[:1], table, free, count, 16)
    with pytest.raises(ValueError):
        fd.reorder_pages(par, lens, table[:1], free, count, 16)
    with pytest.raises(ValueError):
        fd.reorder_pages(par, lens, table, free, count, 16, copies=_i32([[0, 0, 0]]))
    with pytest.raises(fd.FDError):
        fd.reorder_pages(par, lens, table, free, count, 0)
    with pytest.raises(fd.FDError):
        fd.reorder_pages(par, lens, table, free, count, 16, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert lens.tolist() == s.lens and table.tolist() == s.table
