"""Page bookkeeping on the GPU (fd_resize_pages) against a stack and plain
loops: exact, lengths of 0 and 1, pages of one token, growth and release in
one call, shortage of pages, of table columns and of slots."""
import random

import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import resize_ref

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


class State:
    """The same pool on the GPU and as lists."""

    def __init__(self, B, page, width, num_pages, seed):
        self.page = page
        rng = random.Random(seed)
        order = list(range(num_pages))
        rng.shuffle(order)
        self.seq, self.table = [0] * B, [[-3] * width for _ in range(B)]
        self.free, self.count = order, num_pages
        self.d_seq, self.d_table = _i32(self.seq), _i32(self.table).reshape(B, width)
        self.d_free, self.d_count = _i32(self.free), _i32([self.count])

    def step(self, target, room=None, tokens=True):
        B = len(self.seq)
        want = resize_ref(self.seq, target, self.table, self.free, self.count, self.page, room)
        size = len(want[4]) + 5 if room is None else room
        slots = torch.full((size,), -9, dtype=torch.int32, device="cuda") if tokens else None
        pos = torch.full((size,), -9, dtype=torch.int32, device="cuda") if tokens else None
        cu = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda") if tokens else None
        got = fd.resize_pages(self.d_seq, _i32(target), self.d_table, self.d_free, self.d_count, self.page,
                              slots=slots, positions=pos, cu_new=cu)
        assert got is cu
        self.seq, self.table, self.free, self.count = want[:4]
        assert self.d_seq.tolist() == self.seq
        assert self.d_table.tolist() == self.table
        assert int(self.d_count) == self.count
        assert self.d_free.tolist()[: self.count] == self.free[: self.count]
        if tokens:
            n = len(want[4])
            assert cu.tolist() == want[6]
            assert slots.tolist() == want[4] + [-1] * (size - n)
            assert pos.tolist() == want[5] + [0] * (size - n)


@pytest.mark.parametrize("B", [1, 2, 33, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [1, 16, 48, 256])
def test_random_walk(B, page):
    """Admissions, steps, rollbacks and ends in one batch, several calls."""
    rng = random.Random(B * 1000 + page)
    width = 6
    s = State(B, page, width, B * 4 + 3, seed=page)
    for _ in range(6):
        target = []
        for n in s.seq:
            target.append(rng.choice([0, n, n + 1, max(0, n - 3), rng.randrange(width * page + 1),
                                      rng.randrange(width * page + 1)]))
        s.step(target)


@pytest.mark.parametrize("page", [1, 16])
def test_release_undoes_growth(page):
    s = State(40, page, 20, 500, seed=1)
    s.step([i % 7 * page for i in range(40)])
    before = (list(s.seq), s.d_free.tolist(), int(s.d_count))
    s.step([n + 2 * page + 1 for n in s.seq])
    s.step(before[0], tokens=False)
    assert (s.d_seq.tolist(), s.d_free.tolist(), int(s.d_count)) == before


def test_shortage_of_pages_serves_the_first_sequences():
    s = State(5, 16, 8, 6, seed=2)
    s.step([33, 32, 20, 10, 0])    # 3 + 2 pages, then none left for 2, one for none
    assert s.seq == [33, 32, 0, 0, 0]
    s.step([34, 0, 20, 10, 0])     # a sequence that needs no page grows; released pages serve this call
    assert s.seq == [34, 0, 20, 10, 0]


def test_shortage_of_columns_and_slots():
    s = State(4, 16, 3, 50, seed=3)
    s.step([48, 49, 47, 1])        # 49 tokens need a fourth column
    assert s.seq == [48, 0, 47, 1]
    s.step([48, 16, 48, 17], room=16)   # 16 + 1 new tokens pass the 16 slots
    assert s.seq == [48, 16, 47, 1]


def test_one_long_request_and_exact_room():
    s = State(1, 16, 9000, 9000, seed=4)
    s.step([9000 * 16], room=9000 * 16)
    s.step([0], tokens=False)
    s.step([1])


def test_outputs_are_optional_and_padded():
    s = State(3, 16, 4, 20, seed=5)
    s.step([5, 0, 17], tokens=False)
    pos = torch.full((64,), -9, dtype=torch.int32, device="cuda")
    cu = fd.resize_pages(s.d_seq, _i32([6, 1, 17]), s.d_table, s.d_free, s.d_count, 16, positions=pos)
    assert cu.tolist() == [0, 1, 2, 2] and pos.tolist() == [5, 0] + [0] * 62


def test_empty_batch():
    s = State(0, 16, 4, 20, seed=6)
    cu = fd.resize_pages(s.d_seq, _i32([]), s.d_table.reshape(0, 4), s.d_free, s.d_count, 16,
                         slots=_i32([5, 5]), cu_new=None)
    assert cu.tolist() == [0] and int(s.d_count) == 20


def test_bad_state_is_reported():
    """A table entry that names no page is released: reported, the rest of the call stands."""
    s = State(2, 16, 4, 8, seed=7)
    s.step([20, 20])
    s.d_table[1, 0] = 99
    fd.resize_pages(s.d_seq, _i32([20, 0]), s.d_table, s.d_free, s.d_count, 16)
    assert fd.device_status() == 7 and s.d_seq.tolist() == [20, 0]
    s = State(1, 16, 4, 2, seed=8)
    s.d_count.fill_(2)
    s.d_seq.fill_(30)            # says it holds two pages, but the stack is full
    s.d_table[0, :2] = 0
    fd.resize_pages(s.d_seq, _i32([0]), s.d_table, s.d_free, s.d_count, 16)
    assert fd.device_status() == 7 and int(s.d_count) == 2


def test_captured_and_replayed():
    s = State(64, 16, 10, 400, seed=9)
    s.step([i for i in range(64)])
    target = torch.empty_like(s.d_seq)
    slots, pos = (torch.empty(64, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = torch.empty(65, dtype=torch.int32, device="cuda")

    def call():
        torch.add(s.d_seq, 1, out=target)
        fd.resize_pages(s.d_seq, target, s.d_table, s.d_free, s.d_count, 16, slots=slots, positions=pos, cu_new=cu)

    keep = [t.clone() for t in (s.d_seq, s.d_table, s.d_free, s.d_count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for t, x in zip((s.d_seq, s.d_table, s.d_free, s.d_count), keep):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(40):
        graph.replay()
        want = resize_ref(s.seq, [n + 1 for n in s.seq], s.table, s.free, s.count, 16)
        s.seq, s.table, s.free, s.count = want[:4]
        assert slots.tolist() == want[4] and pos.tolist() == want[5] and cu.tolist() == want[6]
    assert s.d_table.tolist() == s.table and int(s.d_count) == s.count
