"""PagePool on a B200 against a host model of the same rules (lists and dicts): table,
lengths, counts, new page numbers and every byte of the pools must be equal."""
import random

import pytest
import torch

from persistent_decode_b200 import PagePool, XlpkError, _abi

pytestmark = pytest.mark.gpu


class Host:
    """The rules of the page operations on host lists."""

    def __init__(self, P, table, lens, refs, k, v):
        self.P, self.table, self.lens, self.refs = P, [list(r) for r in table], list(lens), list(refs)
        self.pools = [k.clone(), v.clone()]

    def free(self):
        return [i for i, n in enumerate(self.refs) if n == 0]

    def fork(self, parents):
        P, rows = self.P, len(self.table)
        free, new, fresh = self.free(), [], 0
        heir = {}
        for r, p in enumerate(parents):
            if p >= 0 and (p not in heir or p == r):
                heir[p] = r
        refs = list(self.refs)
        for r in range(rows):
            for e in self.table[r]:
                if 0 <= e < len(refs):
                    refs[e] -= 1
        for r, p in enumerate(parents):
            row = [-1] * len(self.table[0])
            if p >= 0:
                full = self.lens[p] // P
                if heir[p] == r:
                    row = list(self.table[p])
                else:
                    row[:full] = self.table[p][:full]
                    if self.lens[p] % P:
                        d, s = free[fresh], self.table[p][full]
                        fresh += 1
                        row[full] = d
                        for pool in self.pools:
                            pool[:, d, :, :self.lens[p] % P] = pool[:, s, :, :self.lens[p] % P]
            new.append(row)
        for row in new:
            for e in row:
                if 0 <= e < len(refs):
                    refs[e] += 1
        self.lens = [self.lens[p] if p >= 0 else 0 for p in parents]
        self.table, self.refs = new, refs

    def reserve(self, want):
        free = iter(self.free())
        for r, w in enumerate(want):
            for j in range(self.lens[r] // self.P, -(-w // self.P)):
                if w > self.lens[r] and not 0 <= self.table[r][j] < len(self.refs):
                    self.table[r][j] = next(free)
                    self.refs[self.table[r][j]] = 1

    def trim(self, window, sinks):
        for r, row in enumerate(self.table):
            for j, e in enumerate(row):
                if window and 0 <= e < len(self.refs) and (j + 1) * self.P <= self.lens[r] - window and j * self.P >= sinks:
                    self.refs[e] -= 1
                    row[j] = -1

    def compact(self):
        n = sum(c > 0 for c in self.refs)
        remap = [i if c > 0 else -1 for i, c in enumerate(self.refs)]
        holes = [i for i in range(n) if self.refs[i] == 0]
        high = [i for i in range(n, len(self.refs)) if self.refs[i] > 0]
        for d, s in zip(holes, high):
            remap[s] = d
            for pool in self.pools:
                pool[:, d] = pool[:, s]
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[remap[e] if 0 <= e < len(self.refs) else e for e in row] for row in self.table]
        return remap


def make(rows, cols, P, n_pages, lens, L=2, KH=2, D=64, dtype=torch.bfloat16, seed=0, share=0):
    g = torch.Generator().manual_seed(seed)
    shape = (L, n_pages, KH, P, D)
    k, v = (torch.randint(0, 256, shape, dtype=torch.uint8, generator=g) if dtype == torch.uint8 else
            torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    ids = torch.randperm(n_pages, generator=g).tolist()
    table, refs = [[-1] * cols for _ in range(rows)], [0] * n_pages
    for r, n in enumerate(lens):
        for j in range(-(-n // P)):
            table[r][j] = table[0][j] if r and j < share and (j + 1) * P <= min(n, lens[0]) else ids.pop()
            refs[table[r][j]] += 1
    h = Host(P, table, lens, refs, k, v)
    i32 = dict(dtype=torch.int32, device="cuda")
    return h, PagePool(k.cuda(), v.cuda(), torch.tensor(table, **i32), torch.tensor(lens, **i32), torch.tensor(refs, **i32))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(h, p):
    assert p.seq_lens.tolist() == h.lens
    assert p.page_table.tolist() == h.table
    assert p.refs.tolist() == h.refs
    for got, want in zip((p.k, p.v), h.pools):
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


def snapshot(p):
    return [t.clone() for t in (p.k, p.v, p.page_table, p.seq_lens, p.refs)]


def unchanged(p, snap):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(snapshot(p), snap))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("P,D", [(16, 64), (7, 64), (1, 128), (64, 128)])
def test_fork(cuda_device, P, D, dtype):
    lens = [0, 1, P, P + 1, 3 * P, 4 * P - 1]
    for parents in ([5, 5, 5, 5, 5, 5], [0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [-1] * 6, [3, 3, 1, 1, -1, 4], [1, 0, 3, 3, 3, -1]):
        h, p = make(6, 5, P, 40, lens, D=D, dtype=dtype, share=1)
        h.fork(parents)
        p.fork(i32(parents))
        p.check()
        same(h, p)


def test_fork_keeps_reserved_pages_with_the_heir(cuda_device):
    h, p = make(3, 6, 8, 20, [11, 5, 0])
    h.reserve([40, 5, 0])
    p.reserve(i32([40, 5, 0]))
    same(h, p)
    h.fork([1, 0, 0])
    p.fork(i32([1, 0, 0]))
    p.check()
    same(h, p)


def test_reserve(cuda_device):
    h, p = make(5, 8, 4, 40, [0, 3, 4, 9, 12])
    for want in ([0, 4, 5, 9, 30], [1, 4, 0, 32, 12], [32, 32, 5, 32, -3]):
        h.reserve(want)
        p.reserve(i32(want))
        p.check()
        same(h, p)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (10, 3), (16, 16), (1000, 2)])
def test_trim_then_compact(cuda_device, window, sinks):
    h, p = make(4, 12, 8, 60, [90, 64, 7, 33], share=2, dtype=torch.uint8)
    h.trim(window, sinks)
    p.trim(window, sinks)
    same(h, p)
    want, remap = h.compact(), p.compact()
    p.check()
    assert remap.tolist() == want
    same(h, p)
    h.reserve([91, 65, 8, 40])     # pages given back are taken again, lowest first
    p.reserve(i32([91, 65, 8, 40]))
    same(h, p)


def test_compact_keeps_the_callers_own_references(cuda_device):
    h, p = make(2, 6, 8, 30, [20, 9], seed=3)
    held = max(h.free())
    h.refs[held] += 1
    p.refs[held] += 1
    want, remap = h.compact(), p.compact()
    same(h, p)
    assert remap.tolist() == want and 0 <= want[held] < sum(c > 0 for c in h.refs)


@pytest.mark.parametrize("empty", [True, False])
def test_compact_with_nothing_to_move(cuda_device, empty):
    h, p = make(2, 6, 8, 30, [0, 0] if empty else [40, 40], seed=4)
    for _ in range(2):
        assert p.compact().tolist() == h.compact()
        same(h, p)


def test_many_rows_and_a_large_pool(cuda_device):
    # 1024 rows and 5000 pages of one position: plans of several stretches, every row forked off one
    rows = 1024
    lens = [2 if r == 0 else (r % 3) for r in range(rows)]
    h, p = make(rows, 9, 2, 5000, lens, L=1, KH=1, seed=5)
    want = [n + 5 for n in lens]
    h.reserve(want)
    p.reserve(i32(want))
    p.check()
    same(h, p)
    parents = [(r * 7) % rows if r % 5 else -1 for r in range(rows)]
    h.fork(parents)
    p.fork(i32(parents))
    p.check()
    same(h, p)
    h.lens[3] = 3
    p.seq_lens[3] = 3
    h.reserve([4 if r == 3 else 0 for r in range(rows)])
    p.reserve(i32([4 if r == 3 else 0 for r in range(rows)]))
    h.fork([3] * rows)
    p.fork(i32([3] * rows))
    p.check()
    same(h, p)
    assert p.compact().tolist() == h.compact()
    same(h, p)


def test_a_long_run_of_random_calls(cuda_device):
    rng = random.Random(7)
    h, p = make(6, 10, 8, 50, [13, 40, 8, 0, 25, 1], seed=6, dtype=torch.uint8)
    for step in range(60):
        op = rng.choice(["fork", "reserve", "trim", "compact"])
        if op == "fork":
            parents = [rng.choice([r, r, rng.randrange(-1, 6)]) for r in range(6)]
            if sum(1 for q in set(parents) if q >= 0) == 0 or len(h.free()) < 6:
                continue
            h.fork(parents)
            p.fork(i32(parents))
        elif op == "reserve":
            want = [min(80, n + rng.choice([0, 1, 9])) for n in h.lens]
            if len(h.free()) < 12:
                continue
            h.reserve(want)
            p.reserve(i32(want))
            # positions are filled: a row with no holes behind its window grows
            h.lens = [max(n, w) for n, w in zip(h.lens, want)]
            p.seq_lens.copy_(i32(h.lens))
        elif op == "trim":
            h.trim(30, 4)
            p.trim(30, 4)
        else:
            assert p.compact().tolist() == h.compact()
        p.check()
        same(h, p)


def test_copy(cuda_device):
    h, p = make(2, 30, 4, 1100, [9, 5], L=1)
    src, dst = list(range(0, 1000, 2)) + [0, 0], list(range(1, 1001, 2)) + [1001, 1099]
    for s, d in zip(src, dst):
        for pool in h.pools:
            pool[:, d] = pool[:, s]
    p.copy(src, dst)
    p.copy([], [])
    same(h, p)
    with pytest.raises(ValueError):
        p.copy([1], [2, 3])
    for s, d in (([1, 2], [3, 3]), ([1], [1100]), ([2, 3], [3, 4])):
        with pytest.raises(XlpkError):
            p.copy(s, d)
    same(h, p)


@pytest.mark.parametrize("what", ["oom", "reserve_oom", "full", "parent", "length", "missing_page", "trim_length"])
def test_what_cannot_be_done_changes_nothing_and_stops_the_pool(cuda_device, what):
    h, p = make(4, 4, 8, 12, [20, 9, 0, 31], seed=9)
    want = _abi.XLPK_ERR_INVALID_ARG
    if what in ("length", "trim_length"):
        p.seq_lens[1] = 33
    if what == "missing_page":
        p.page_table[1, 1] = -1
    snap = snapshot(p)
    if what == "oom":
        p.refs += 1        # every page is held
        snap = snapshot(p)
        p.fork(i32([0, 0, 0, 3]))
        want = _abi.XLPK_ERR_OOM
    elif what == "reserve_oom":
        p.reserve(i32([32, 32, 32, 32]))     # 5 pages lack, 3 are free
        want = _abi.XLPK_ERR_OOM
    elif what == "full":
        p.reserve(i32([20, 33, 0, 31]))
        want = _abi.XLPK_ERR_KV_FULL
    elif what == "parent":
        p.fork(i32([0, 4, 2, 3]))
    elif what == "trim_length":
        p.trim(1)
    else:
        p.fork(i32([1, 1, 2, 3]))
    # later calls wait for the caller
    p.fork(i32([-1] * 4))
    p.reserve(i32([21, 10, 1, 32]))
    p.trim(1)
    p.compact()
    p.copy([0], [1])
    assert unchanged(p, snap)
    with pytest.raises(XlpkError) as e:
        p.check()
    assert e.value.status == want
    p.check()
    p.copy([0], [1])
    assert not unchanged(p, snap)


def test_compact_of_a_stopped_pool_returns_the_numbers_that_pages_have(cuda_device):
    h, p = make(4, 6, 8, 3000, [20, 9, 0, 31], L=1, seed=18)
    snap = snapshot(p)
    p.fork(i32([0, 0, 0, 9]))          # no such row
    junk = torch.full((3000,), 12345, dtype=torch.int32, device=cuda_device)
    del junk                           # what the result's memory may have held
    remap = p.compact()
    assert remap.tolist() == [i if c > 0 else -1 for i, c in enumerate(h.refs)]
    assert unchanged(p, snap)
    with pytest.raises(XlpkError):
        p.check()
    assert p.compact().tolist() == h.compact()
    same(h, p)


@pytest.mark.parametrize("row", [0, 255, 256, 511, 700, 999])
def test_trim_of_a_large_table_changes_all_or_nothing(cuda_device, row):
    # a table of hundreds of CTAs' work with one bad length: whichever thread looks at it, and however
    # late a CTA starts, nothing is trimmed; with the length put right everything behind the window is
    rows, cols, P, pages = 1000, 600, 2, 64
    g = torch.Generator().manual_seed(row)
    table = torch.randint(0, pages, (rows, cols), generator=g, dtype=torch.int32)
    lens = torch.randint(0, cols * P + 1, (rows,), generator=g, dtype=torch.int32)
    k = torch.zeros((1, pages, 1, P, 64), dtype=torch.bfloat16, device=cuda_device)
    p = PagePool(k, k.clone(), table.cuda(), lens.cuda())
    snap = snapshot(p)
    for bad in (-1, cols * P + 1) * 10:
        p.seq_lens[row] = bad
        p.trim(100, 7)
        with pytest.raises(XlpkError) as e:
            p.check()
        assert e.value.status == _abi.XLPK_ERR_INVALID_ARG
        p.seq_lens[row] = lens[row]
        assert unchanged(p, snap)
    p.trim(100, 7)
    p.check()
    j = torch.arange(cols)
    gone = ((j + 1) * P <= lens[:, None] - 100) & (j * P >= 7)
    want = torch.where(gone, -1, table)
    assert torch.equal(p.page_table.cpu(), want)
    assert torch.equal(p.refs.cpu(), torch.bincount(want[want >= 0].long(), minlength=pages).int())


def test_assigned_tensors_are_used_and_bad_ones_refused(cuda_device):
    h, p = make(4, 6, 8, 40, [20, 9, 0, 31], seed=20)
    p.seq_lens = p.seq_lens + 1                    # the tensor before has no owner any more:
    others = [torch.full((4,), -7, dtype=torch.int32, device=cuda_device) for _ in range(64)]   # its memory is theirs
    h.lens = [n + 1 for n in h.lens]
    h.reserve([21, 10, 1, 32])
    p.reserve(i32([21, 10, 1, 32]))
    p.check()
    same(h, p)
    p.page_table, p.refs = p.page_table.clone(), p.refs.clone()
    p.k, p.v = p.k.clone(), p.v.clone()
    p.status = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    others += [torch.full_like(t, -7) for t in (p.page_table, p.refs) for _ in range(16)]
    h.fork([0, 0, 1, 3])
    p.fork(i32([0, 0, 1, 3]))
    assert p.compact().tolist() == h.compact()
    p.check()
    same(h, p)
    p.seq_lens += 1                                # in place, and assigned
    p.refs[:1] += 0
    h.lens = [n + 1 for n in h.lens]
    same(h, p)
    p.seq_lens.data = p.seq_lens.clone()           # the same tensor at another address
    others += [torch.full((4,), -7, dtype=torch.int32, device=cuda_device) for _ in range(64)]
    h.reserve([30, 30, 30, 40])
    p.reserve(i32([30, 30, 30, 40]))
    p.check()
    same(h, p)
    for t in others:
        assert bool((t == -7).all())
    for name, bad in (("seq_lens", p.seq_lens[:3]), ("seq_lens", p.seq_lens.long()), ("seq_lens", p.seq_lens.cpu()), ("seq_lens", None),
                      ("page_table", p.page_table[:2]), ("page_table", p.page_table[:, ::2]), ("refs", p.refs[:5]),
                      ("k", p.k[:, :4]), ("v", p.v.view(torch.uint8)), ("status", p.status[:0])):
        was = getattr(p, name)
        with pytest.raises(ValueError):
            setattr(p, name, bad)
        assert getattr(p, name) is was
    h.fork([3, 0, 1, 3])
    p.fork(i32([3, 0, 1, 3]))
    p.check()
    same(h, p)


def test_captured_and_replayed(cuda_device):
    h, p = make(4, 6, 8, 40, [20, 9, 0, 31], seed=10)
    parents, want = i32([0, 0, 1, 3]), i32([24, 24, 16, 32])
    side = make(4, 6, 8, 40, [20, 9, 0, 31], seed=11)[1]
    side.fork(parents)
    side.reserve(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.fork(parents)
        p.reserve(want)
        p.trim(8, 4)
        remap = p.compact()
    same(h, p)             # recorded, not run
    for par, w in (([0, 0, 1, 3], [24, 24, 16, 32]), ([3, 0, 1, 1], [33, 0, 24, 17])):
        parents.copy_(i32(par))
        want.copy_(i32(w))
        g.replay()
        h.fork(par)
        h.reserve(w)
        h.trim(8, 4)
        assert remap.tolist() == h.compact()
        p.check()
        same(h, p)


def test_on_another_stream(cuda_device):
    h, p = make(3, 6, 8, 40, [20, 9, 31], seed=12)
    st = torch.cuda.Stream()
    parents = i32([2, 0, 2])
    torch.cuda.synchronize()
    p.fork(parents, stream=st)
    remap = p.compact(stream=st)
    st.synchronize()
    h.fork([2, 0, 2])
    assert remap.tolist() == h.compact()
    same(h, p)


@pytest.mark.parametrize("how", ["argument", "context"])
def test_check_waits_for_every_stream(cuda_device, how):
    # calls on two side streams, each behind some milliseconds of other work, and no other synchronisation
    h, p = make(4, 4, 8, 12, [20, 9, 0, 31], seed=13)
    snap = snapshot(p)
    busy = torch.randn(4096, 4096, device=cuda_device)
    want = i32([32, 32, 32, 32])        # 5 pages lack, 3 are free
    fits = i32([24, 16, 8, 32])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()

    def reserve(st, w):
        with torch.cuda.stream(st):
            for _ in range(30):
                torch.mm(busy, busy)
            if how == "context":
                p.reserve(w)
        if how == "argument":
            p.reserve(w, stream=st)

    for bad in streams:
        reserve(bad, want)
        with pytest.raises(XlpkError) as e:
            p.check()
        assert e.value.status == _abi.XLPK_ERR_OOM
        assert unchanged(p, snap)
        p.check()
    for _ in range(30):                 # the other way round: from a side stream, a call on the default one
        torch.mm(busy, busy)
    p.reserve(want)
    with torch.cuda.stream(streams[0]):
        with pytest.raises(XlpkError):
            p.check()
    # the status is clear for the next call of another stream, which check() waits for as well
    reserve(streams[0], fits)
    p.check()
    h.reserve([24, 16, 8, 32])
    same(h, p)


def test_check_while_another_stream_records(cuda_device):
    h, p = make(3, 6, 8, 40, [20, 9, 31], seed=14)
    p.fork(i32([0, 1, 2]))
    st, parents = torch.cuda.Stream(), i32([2, 0, 2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        g.capture_begin(capture_error_mode="relaxed")
        p.fork(parents)
    p.check()
    with torch.cuda.stream(st):
        g.capture_end()
        g.replay()
    p.check()              # (the graph was replayed on the stream that recorded it)
    h.fork([2, 0, 2])
    same(h, p)


def test_offsets_past_32_bits(cuda_device):
    # one layer of K and V of more than 2^32 bytes each; pages at its end are copied, forked and moved to its start
    P, n = 1024, (1 << 32) // (1024 * 128) + 64
    k, v = (torch.empty((1, n, 1, P, 128), dtype=torch.uint8, device=cuda_device) for _ in range(2))
    refs = torch.zeros(n, dtype=torch.int32, device=cuda_device)
    refs[n - 2:] = 1
    g = torch.Generator(device=cuda_device).manual_seed(1)
    for t in (k, v):
        t[:, n - 2:] = torch.randint(0, 256, t[:, n - 2:].shape, dtype=torch.uint8, generator=g, device=cuda_device)
    full, part = [t[0, n - 2].clone() for t in (k, v)], [t[0, n - 1].clone() for t in (k, v)]
    table, lens = i32([[n - 2, n - 1, -1], [-1, -1, -1]]), i32([P + 700, 0])
    p = PagePool(k, v, table, lens, refs)
    p.copy([n - 2], [n - 3])
    p.fork(i32([0, 0]))
    p.check()
    assert table.tolist() == [[n - 2, n - 1, -1], [n - 2, 0, -1]]
    for t, f, q in zip((k, v), full, part):
        assert torch.equal(t[0, n - 3], f) and torch.equal(t[0, 0, :, :700], q[:, :700])
    remap = p.compact()
    p.check()
    assert table.tolist() == [[1, 2, -1], [1, 0, -1]] and remap[n - 2:].tolist() == [1, 2]
    for t, f, q in zip((k, v), full, part):
        assert torch.equal(t[0, 1], f) and torch.equal(t[0, 2], q)


def test_refusals(cuda_device):
    h, p = make(2, 4, 8, 12, [20, 9])
    k, v, t, n, r = p.k, p.v, p.page_table, p.seq_lens, p.refs
    for bad in (lambda: PagePool(k.float(), v.float(), t, n, r), lambda: PagePool(k, v[:1], t, n, r),
                lambda: PagePool(k.transpose(2, 3), v.transpose(2, 3), t, n, r), lambda: PagePool(k, v, t.long(), n, r),
                lambda: PagePool(k, v, t[:, ::2], n, r), lambda: PagePool(k, v, t, n[:1], r), lambda: PagePool(k, v, t, n, r[:5]),
                lambda: PagePool(k, v, t, n.cpu(), r), lambda: p.fork(i32([0])), lambda: p.fork(i32([0, 1]).long()),
                lambda: p.reserve(i32([1, 2, 3])), lambda: p.reserve(torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(XlpkError):
        p.trim(-1)
    assert PagePool(k, v, t, n).refs.tolist() == h.refs
    same(h, p)
