"""The serving path as it is used: pages reserved, rows appended, new tokens
attended (chunks of prompts, drafted tokens, rejected drafts given back,
single tokens through decode), checked against attention over each request's
whole history in float64."""
import pytest
import torch

import split_kv_fd_gb300 as fd
from serve_util import attend, check

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


class Server:
    def __init__(self, B, page, num_pages, Hq, Hkv, d, dtype, fp8):
        self.B, self.page, self.Hq, self.Hkv, self.d, self.dtype, self.fp8 = B, page, Hq, Hkv, d, dtype, fp8
        kind = torch.float8_e4m3fn if fp8 else dtype
        self.kp, self.vp = (torch.zeros(num_pages, Hkv, page, d, dtype=torch.uint8 if fp8 else dtype, device="cuda").view(kind)
                            for _ in range(2))
        self.table = torch.full((B, 64), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(num_pages, device="cuda").to(torch.int32)
        self.count, self.seq = _i32([num_pages]), _i32([0] * B)
        self.ks, self.vs = (torch.rand(B, Hkv, device="cuda") * 0.01 + 0.01 for _ in range(2))
        self.hist = [[torch.zeros(0, Hkv, d, dtype=torch.float64, device="cuda")] * 2 for _ in range(B)]

    def stored(self, x, scale):
        """What the cache holds of a row."""
        if not self.fp8:
            return x.double()
        q = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return q.double() * scale.double()[:, None]

    def step(self, new, decode=False):
        old = self.seq.tolist()
        T = sum(new) + 3    # a padded batch
        qkv = torch.randn(T, self.Hq + 2 * self.Hkv, self.d, device="cuda").to(self.dtype)
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
        slots = torch.empty(T, dtype=torch.int32, device="cuda")
        pos = torch.empty_like(slots)
        cu = fd.resize_pages(self.seq, _i32([o + n for o, n in zip(old, new)]), self.table, self.free, self.count, self.page,
                             slots=slots, positions=pos)
        if self.fp8:
            fd.append_paged_fp8(k, v, self.ks, self.vs, cu, slots, self.kp, self.vp)
        else:
            fd.append_paged(k, v, slots, self.kp, self.vp)
        assert self.seq.tolist() == [o + n for o, n in zip(old, new)]
        if decode:
            qd = q[: self.B].contiguous()
            if self.fp8:
                out, lse = fd.decode_gqa_paged_fp8(qd, self.kp, self.vp, self.ks, self.vs, self.table, self.seq,
                                                   out_dtype=torch.float32)
            else:
                out, lse = fd.decode_gqa_paged(qd, self.kp, self.vp, self.table, self.seq, out_dtype=torch.float32)
        elif self.fp8:
            out, lse = fd.extend_paged_fp8(q, self.kp, self.vp, self.ks, self.vs, self.table, cu, self.seq,
                                           out_dtype=torch.float32)
        else:
            out, lse = fd.extend_paged(q, self.kp, self.vp, self.table, cu, self.seq, out_dtype=torch.float32)
        at = 0
        for b, n in enumerate(new):
            rows = slice(at, at + n)
            at += n
            self.hist[b] = [torch.cat([h, self.stored(x[rows], s[b])])
                            for h, x, s in zip(self.hist[b], (k, v), (self.ks, self.vs))]
            if n:
                check(out[rows], lse[rows], attend(q[rows], *self.hist[b]), self.dtype, old[b] + n, f"request {b}")

    def cut(self, lens):
        fd.resize_pages(self.seq, _i32(lens), self.table, self.free, self.count, self.page)
        assert self.seq.tolist() == lens
        self.hist = [[x[:n] for x in h] for h, n in zip(self.hist, lens)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,dtype", [(16, torch.bfloat16), (64, torch.float16)])
def test_a_serving_loop(fp8, page, dtype):
    torch.manual_seed(page)
    s = Server(4, page, 200, 8, 2, 128, dtype, fp8)
    s.step([70, 0, 5, 300])           # prompts
    s.step([130, 33, 1, 0])           # a second chunk, an admission, a single token
    s.step([1, 1, 1, 1], decode=True)
    s.step([4, 4, 4, 4])              # drafts
    s.cut([n - r for n, r in zip(s.seq.tolist(), (3, 0, 1, 4))])   # rejected ones
    s.step([1, 1, 1, 1], decode=True)
    s.cut([0, s.seq.tolist()[1], 0, s.seq.tolist()[3]])            # two requests end
    s.step([200, 2, 17, 2])           # their pages serve new ones
    s.cut([0] * 4)
    assert int(s.count) == 200 and sorted(s.free.tolist()) == list(range(200))


def test_prefill_is_the_first_chunk():
    """A prompt attended packed and the same rows attended over the cache they were appended to."""
    lens, Hq, Hkv, d, page = [150, 1, 700], 8, 2, 128, 32
    qkv = torch.randn(sum(lens), Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kp, vp = (torch.zeros(40, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, seq = torch.zeros(3, 25, dtype=torch.int32, device="cuda"), _i32([0, 0, 0])
    slots = torch.empty(sum(lens), dtype=torch.int32, device="cuda")
    cu = fd.resize_pages(seq, _i32(lens), table, torch.arange(40, dtype=torch.int32, device="cuda"), _i32([40]), page, slots=slots)
    fd.append_paged(k, v, slots, kp, vp)
    a = fd.extend_paged(q, kp, vp, table, cu, seq, out_dtype=torch.float32)
    b = fd.prefill(q, k, v, cu, out_dtype=torch.float32)
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        ref = attend(q[rows], k[rows], v[rows])
        check(a[0][rows], a[1][rows], ref, torch.bfloat16, n)
        check(b[0][rows], b[1][rows], ref, torch.bfloat16, n)


def test_a_captured_step():
    """Bookkeeping, append and attention in one graph, replayed with new
    targets and rows; a second graph uses the same workspace in turn."""
    B, page, pool, Hq, Hkv, d, width, T = 5, 32, 60, 8, 2, 64, 12, 96
    torch.manual_seed(4)
    kp, vp = (torch.full((pool, Hkv, page, d), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count, seq, target = torch.randperm(pool, device="cuda").to(torch.int32), _i32([pool]), _i32([0] * B), _i32([0] * B)
    qkv = torch.zeros(T, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    slots, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fd.workspace_size_extend(B, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(T, Hq, d, device="cuda") for _ in range(2)]
    lses = [torch.zeros(T, Hq, device="cuda") for _ in range(2)]

    def step(i):
        fd.resize_pages(seq, target, table, free, count, page, slots=slots, positions=pos, cu_new=cu)
        fd.append_paged(k, v, slots, kp, vp)
        fd.extend_paged(q, kp, vp, table, cu, seq, out=outs[i], lse=lses[i], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)   # nothing grows: every target is 0
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            step(i)
    hist = [[torch.zeros(0, Hkv, d, dtype=torch.float64, device="cuda")] * 2 for _ in range(B)]
    old = [0] * B
    for i, want in enumerate([[40, 0, 1, 33, 20], [41, 1, 2, 34, 21], [41, 80, 2, 38, 0], [45, 81, 0, 39, 60], [50, 90, 9, 0, 90]]):
        target.copy_(_i32(want))
        qkv.normal_()
        outs[i % 2].fill_(5)
        graphs[i % 2].replay()
        assert seq.tolist() == want
        at = 0
        for b in range(B):
            n = max(0, want[b] - old[b])
            rows = slice(at, at + n)
            at += n
            hist[b] = [torch.cat([h, x[rows].double()])[: want[b]] for h, x in zip(hist[b], (k, v))]
            assert pos[rows].tolist() == list(range(old[b], old[b] + n))
            check(outs[i % 2][rows], lses[i % 2][rows], attend(q[rows], *hist[b]), torch.bfloat16, want[b], f"request {b}")
        assert bool((outs[i % 2][at:] == 5).all()) and bool((slots[at:] == -1).all())
        old = want
