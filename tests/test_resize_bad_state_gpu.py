"""Page bookkeeping whose state is wrong: ids that name no page, a stack that
would overflow.  Nothing of it may reach another sequence's pages."""
import pytest
import torch

import split_kv_fd_gb300 as fd

pytestmark = pytest.mark.gpu

BAD_PAGE = 7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ids whose product with a page of 256 tokens passes 2^31 or 2^32 and comes
# back into the pool, one just behind it, and negative ones
BAD_IDS = [0x01000005, 0x00800003, 8, 99, -1, -(1 << 31), (1 << 31) - 1]


@pytest.mark.parametrize("room", [300, 3000])
@pytest.mark.parametrize("bad", BAD_IDS)
def test_released_and_taken_in_one_call(bad, room):
    """Sequence 0 releases page 2 and an id that is none, sequence 1 takes both."""
    seq, table = _i32([300, 0]), _i32([[2, bad, -1], [-1, -1, -1]])
    free, count = _i32([7, 6, 5, 4, 3, 1, -1, -1]), _i32([0])
    slots, pos = (torch.full((room,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = fd.resize_pages(seq, _i32([0, 300]), table, free, count, 256, slots=slots, positions=pos)
    assert fd.device_status() == BAD_PAGE
    assert seq.tolist() == [0, 300] and cu.tolist() == [0, 0, 300] and int(count) == 0
    assert table[1].tolist() == [2, -1, -1]
    assert slots.tolist() == list(range(512, 768)) + [-1] * (room - 256)
    assert pos.tolist() == list(range(300)) + [0] * (room - 300)


@pytest.mark.parametrize("bad", BAD_IDS)
def test_released_now_and_taken_later(bad):
    seq, table = _i32([300, 0]), _i32([[2, bad], [-1, -1]])
    free, count = _i32([7, 6, 5, 4, -1, -1, -1, -1]), _i32([1])
    fd.resize_pages(seq, _i32([0, 0]), table, free, count, 256)
    assert fd.device_status() == BAD_PAGE
    assert int(count) == 3 and free.tolist()[:3] == [7, -1, 2]
    slots = torch.full((512,), -9, dtype=torch.int32, device="cuda")
    fd.resize_pages(seq, _i32([0, 512]), table, free, count, 256, slots=slots)
    assert fd.device_status() == BAD_PAGE, "taking it is reported too"
    assert slots.tolist() == list(range(512, 768)) + [-1] * 256
    fd.resize_pages(seq, _i32([200, 512]), table, free, count, 256, slots=slots)
    assert fd.device_status() == 0, "the good page below it is served"
    assert slots.tolist() == list(range(7 * 256, 7 * 256 + 200)) + [-1] * 312


@pytest.mark.parametrize("bad", BAD_IDS)
def test_growth_inside_a_page_that_is_none(bad):
    """The table's own entry for a sequence's last page names no page."""
    seq, table = _i32([10, 5]), _i32([[bad], [4]])
    free, count = _i32([0] * 8), _i32([0])
    slots = torch.full((8,), -9, dtype=torch.int32, device="cuda")
    fd.resize_pages(seq, _i32([12, 6]), table, free, count, 256, slots=slots)
    assert fd.device_status() == BAD_PAGE
    assert slots.tolist() == [-1, -1, 4 * 256 + 5] + [-1] * 5


def test_no_other_sequences_rows_are_overwritten():
    """The append behind it leaves the pool's other pages as they were."""
    seq, table = _i32([0, 256]), _i32([[-1], [5]])
    free, count = _i32([0x01000005] + [0] * 7), _i32([1])
    slots = torch.empty(4, dtype=torch.int32, device="cuda")
    fd.resize_pages(seq, _i32([4, 256]), table, free, count, 256, slots=slots)
    pages = [torch.full((8, 1, 256, 64), 7.0, device="cuda") for _ in range(2)]
    rows = torch.ones(4, 1, 64, device="cuda")
    fd.append_paged(rows, rows, slots, *pages)
    assert fd.device_status() == BAD_PAGE
    assert all(bool((p == 7).all()) for p in pages)


@pytest.mark.parametrize("B", [3, 1500])
@pytest.mark.parametrize("extra", [1, 2])
def test_a_stack_that_would_overflow_still_serves(B, extra):
    """More pages come back than the pool has room for: the stack keeps its
    num_pages entries, and growth in the same call takes real ones."""
    seq, table = _i32([0] * B), _i32([[-1, -1]] * B)
    seq[0] = 16 * extra
    table[0, :extra] = _i32([3, 2][:extra])         # pages that are free already
    free, count = _i32([0, 1, 2, 3, 4, 5, 6, 7]), _i32([8])
    target, slots = _i32([0] * B), torch.full((20,), -9, dtype=torch.int32, device="cuda")
    target[B - 1] = 20
    fd.resize_pages(seq, target, table, free, count, 16, slots=slots)
    assert fd.device_status() == BAD_PAGE
    assert seq.tolist() == [0] * (B - 1) + [20]
    assert table[B - 1].tolist() == [7, 6] and int(count) == 6
    assert slots.tolist() == [7 * 16 + i for i in range(16)] + [6 * 16 + i for i in range(4)]
    assert free.tolist() == list(range(8))


def test_an_overflow_drops_what_passes_the_end():
    """One place is left for the three pages of two sequences: the last one's."""
    seq, table = _i32([32, 16, 0]), _i32([[4, 5], [6, -1], [-1, -1]])
    free, count = _i32([0, 1, 2, 3, 7, 1, 2, -1]), _i32([7])
    fd.resize_pages(seq, _i32([0, 0, 0]), table, free, count, 16)
    assert fd.device_status() == BAD_PAGE
    assert int(count) == 8 and free.tolist() == [0, 1, 2, 3, 7, 1, 2, 6]


def test_releases_past_32_bits():
    """1024 sequences that claim 2^22 pages each, 2^32 in all: the counts are
    kept in 64 bits, and the pool of 8 takes its 8."""
    B, width = 1024, 1 << 22
    seq = torch.full((B,), width, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    table[B - 1, width - 8:] = _i32(list(range(8)))
    free, count = _i32([-1] * 8), _i32([0])
    fd.resize_pages(seq, _i32([0] * B), table, free, count, 1)
    assert fd.device_status() == BAD_PAGE
    assert not bool(seq.any()) and int(count) == 8
    assert free.tolist() == [7, 6, 5, 4, 3, 2, 1, 0]
