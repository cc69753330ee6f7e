"""Which requests fd_reorder_pages grants when pages are few, by arithmetic."""
import random

import pytest
import torch

import split_kv_fd_gb300 as fd
from beam_util import BeamPool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__ as g
    g.build()
    fd.load()
    yield
    assert fd.device_status() == 0


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 7, 17, 18, 20])
def test_starts_are_granted_in_order(spare):
    """Six prompts to four beams each: three copies a request and nothing that
    comes back, so the i-th is granted while 3 (i + 1) pages are free."""
    s = BeamPool(random.Random(spare), 6, 4, 16, 4, (20, 20), (0, 0), spare=spare)
    for b in range(24):
        if b % 4:
            s.lens[b] = 0
    lens, table, free, count = s.tensors()
    assert int(count) == spare
    parents = torch.zeros(6, 4, dtype=torch.int32, device="cuda")
    copies, granted = fd.reorder_pages(parents, lens, table, free, count, 16)
    want = [int(3 * (i + 1) <= spare) for i in range(6)]
    assert granted.tolist() == want and int(count) == spare - 3 * sum(want)
    assert lens.tolist() == [20 if w == 0 or want[r] else 0 for r in range(6) for w in range(4)]
    assert [c[2] for c in copies.tolist()] == [4 if w and want[r] else 0 for r in range(6) for w in range(4)]


@pytest.mark.parametrize("spare", [0, 3, 7])
def test_what_others_leave_over_counts(spare):
    """One of the requests ends and gives its two pages back: it is granted, and
    so are those in order whose needs fit what is free and those two."""
    s = BeamPool(random.Random(spare), 6, 4, 16, 4, (20, 20), (0, 0), spare=spare)
    for b in range(24):
        if b % 4:
            s.lens[b] = 0
    for end in (0, 3, 5):
        lens, table, free, count = s.tensors()
        parents = torch.zeros(6, 4, dtype=torch.int32, device="cuda")
        parents[end] = -1
        _, granted = fd.reorder_pages(parents, lens, table, free, count, 16)
        others = [r for r in range(6) if r != end]
        want = [1 if r == end else int(3 * (others.index(r) + 1) <= spare + 2) for r in range(6)]
        assert granted.tolist() == want and int(count) == spare + 2 - 3 * (sum(want) - 1)
