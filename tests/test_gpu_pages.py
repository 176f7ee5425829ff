"""Pages, positions and slots from request lengths (dflash_pages_*) against a
plain Python simulation: whole numbers, compared exactly."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_draft_tcgen05_gb300 import build
    build.build()
    import speculative_decoding_draft_tcgen05_gb300 as p
    p.lib()
    return p


def dev(x, dtype=torch.int32):
    return torch.tensor(x, device="cuda", dtype=dtype)


class Model:
    """A pool as plain lists."""

    def __init__(self, requests, cols, num_pages, page):
        self.table = [[-1] * cols for _ in range(requests)]
        self.lens, self.free, self.page, self.cols, self.requests = [0] * requests, list(range(num_pages - 1, -1, -1)), page, cols, requests

    def need(self, n):
        return -(-n // self.page)

    def extend(self, rows, new, tokens, room=None):
        """cu_tokens, lengths, granted, positions, slots; the requests' rows are in `table`."""
        room = min(self.cols, room or self.cols)
        cu, lens, granted, positions, slots = [0], [], [], [], []
        pages = count = 0
        full = False
        for r, n in zip(rows, new):
            known = 0 <= r < self.requests
            old = self.lens[r] if known else 0
            good = known and n >= 0 and old + n <= room * self.page
            if good:
                pages += self.need(old + n) - self.need(old)
                count += n
            full = full or pages > self.free_at_start(granted) or count > tokens
            ok = good and not full
            if ok:
                for at in range(old, old + n):
                    if at % self.page == 0:
                        self.table[r][at // self.page] = self.free.pop()
                    positions.append(at)
                    slots.append(self.table[r][at // self.page] * self.page + at % self.page)
                self.lens[r] = old + n
            granted.append(int(ok))
            lens.append(self.lens[r] if known else 0)
            cu.append(len(positions))
        return cu, lens, granted, positions, slots

    def free_at_start(self, granted):
        if not granted:
            self.start = len(self.free)
        return self.start

    def trim(self, rows, drop):
        back = []
        for r, d in zip(rows, drop):
            if not 0 <= r < self.requests:
                continue
            d = max(0, min(d, self.lens[r]))
            kept = self.need(self.lens[r] - d)
            back += self.table[r][kept:self.need(self.lens[r])]
            self.lens[r] -= d
        self.free += reversed(back)


class Both:
    """The model and the pool on the GPU, which have to agree after every call."""

    def __init__(self, pkg, requests, cols, num_pages, page, stride=0):
        self.m = Model(requests, cols, num_pages, page)
        self.pool = pkg.PagePool.empty(requests=requests, cols=cols, num_pages=num_pages, page_size=page)
        if stride:
            wide = torch.full((requests, cols + stride), -1, device="cuda", dtype=torch.int32)
            self.pool = pkg.PagePool(wide[:, :cols], self.pool.lens, self.pool.free_pages, self.pool.counters, page_size=page)
        self.pkg = pkg

    def extend(self, new, rows=None, tokens=None, cols=None, own=False):
        m, b = self.m, len(new)
        cap = sum(n for n in new if n > 0) if tokens is None else tokens
        table = self.pool.page_table[:b] if own else torch.full((b, cols or m.cols), -7, device="cuda", dtype=torch.int32)
        lens = self.pool.lens[:b] if own else torch.full((b,), -7, device="cuda", dtype=torch.int32)
        cu = torch.full((b + 1,), -7, device="cuda", dtype=torch.int32)
        batch = self.pkg.PagedBatch(cu, lens, table, max_tokens=max(new + [0]))
        pos, slots = torch.full((cap + 3,), -7, device="cuda", dtype=torch.int32), torch.full((cap + 3,), -7, device="cuda", dtype=torch.int64)
        granted = torch.full((b,), -7, device="cuda", dtype=torch.int32)
        self.pool.extend(batch, dev(new), rows=None if rows is None else dev(rows), positions=pos, slots=slots, granted=granted, tokens=cap)
        rows = list(range(b)) if rows is None else rows
        want = m.extend(rows, new, cap, cols)
        n = want[0][-1]
        assert cu.tolist() == want[0] and lens.tolist() == want[1] and granted.tolist() == want[2]
        assert pos.tolist() == want[3] + [-7] * (cap + 3 - n) and slots.tolist() == want[4] + [-7] * (cap + 3 - n)
        if not own:
            for i, (r, length) in enumerate(zip(rows, want[1])):
                entries = min(m.need(length), table.shape[1])
                assert table[i].tolist() == (m.table[r][:entries] if 0 <= r < m.requests else []) + [-7] * (table.shape[1] - entries)
        self.agree()
        return want

    def trim(self, drop, rows=None):
        self.pool.trim(dev(drop), rows=None if rows is None else dev(rows))
        self.m.trim(range(len(drop)) if rows is None else rows, drop)
        self.agree()

    def agree(self):
        m = self.m
        count = len(m.free)
        assert self.pool.counters.tolist() == [count, 0] and self.pool.lens.tolist() == m.lens
        assert self.pool.free_pages.tolist()[:count] == m.free
        table = self.pool.page_table.tolist()
        held = [p for r in range(m.requests) for p in table[r][:m.need(m.lens[r])]]
        assert all(table[r][:m.need(m.lens[r])] == m.table[r][:m.need(m.lens[r])] for r in range(m.requests))
        assert sorted(held + m.free) == list(range(self.pool.free_pages.shape[0]))  # every page is in one place


@pytest.mark.parametrize("page,requests,batch,most", [(16, 1, 1, 8), (16, 5, 3, 40), (1, 7, 7, 5), (64, 300, 256, 16), (48, 40, 33, 900)])
def test_steps_of_a_server(pkg, page, requests, batch, most):
    r = random.Random(page * requests)
    both = Both(pkg, requests, cols=3 * (most // page + 2), num_pages=requests * (most // page + 2) + 3, page=page, stride=page % 3)
    for step in range(12):
        rows = r.sample(range(requests), batch)
        both.extend([r.choice([0, 1, 1, most, r.randint(0, most)]) for _ in rows], rows)
        both.trim([r.choice([0, 1, r.randint(0, most), 10 ** 6, -3]) for _ in rows], rows)
        if step % 3 == 2:
            both.trim([r.randint(0, 3 * most) for _ in range(requests)])


def test_the_pools_own_tensors(pkg):
    both = Both(pkg, 6, 10, 40, 16)
    both.extend([5, 16, 0, 33, 1, 100], own=True)
    both.extend([30, 1], own=True)
    both.trim([7, 17, 5])
    both.extend([7, 17, 16, 0, 0, 60], own=True)


def test_refused_entries(pkg):
    both = Both(pkg, 8, cols=6, num_pages=12, page=16)
    # a row out of range, a negative number, more than a row of the table holds: refused on their own account
    assert both.extend([3, 5, -1, 97, 2, 96], [0, 9, 1, 2, -1, 3])[2] == [1, 0, 0, 0, 0, 1]
    # 5 pages are left: the third entry does not fit, and what follows it is refused too
    assert both.extend([40, 20, 16, 1, 0], [4, 5, 6, 0, 7])[2] == [1, 1, 0, 0, 0]
    assert both.extend([5], [0])[2] == [1]           # (into its page)
    assert both.extend([1, 9, 1], [0, 1, 4], tokens=5)[2] == [1, 0, 0]  # rows of the batch
    both.trim([10 ** 6] * 8)
    assert both.extend([60, 1], [0, 1], cols=3)[2] == [0, 1]  # a narrower table of the batch
    assert both.extend([48, 1], [0, 1], cols=3)[2] == [1, 1]


@pytest.mark.parametrize("batch", [1023, 1024, 1025, 3000])
def test_large_batches(pkg, batch):
    r = random.Random(batch)
    both = Both(pkg, batch + 5, cols=8, num_pages=4 * batch, page=16)
    rows = r.sample(range(batch + 5), batch)
    both.extend([r.randint(0, 40) for _ in rows], rows)
    both.extend([r.randint(0, 60) for _ in rows], rows)         # the pages run out on the way
    both.trim([r.randint(0, 50) for _ in rows], rows)
    both.extend([1] * batch, rows, tokens=batch // 2)           # the rows do
    both.trim([r.randint(0, 50) for _ in rows], rows)


def test_a_long_prompt(pkg):
    both = Both(pkg, 3, cols=1200, num_pages=2000, page=16)
    both.extend([16001, 0, 700])
    both.extend([8, 8, 8], [2, 0, 1])
    both.trim([15990, 3], [0, 2])


@pytest.mark.parametrize("requests", [1, 40, 300])
def test_thousands_of_pages_move_at_once(pkg, requests):
    """Without positions and slots, a call's blocks share its pages all the same; a trim's as well."""
    r = random.Random(requests)
    cols = 12000 // requests + 3
    m = Model(requests, cols, 12000, 2)
    pool = pkg.PagePool.empty(requests=requests, cols=cols, num_pages=12000, page_size=2)
    rows = r.sample(range(requests), requests)
    new = [2 * cols - 7 + r.randint(0, 3) for _ in rows]
    for drop in ([r.randint(0, 2 * cols) for _ in rows], [10 ** 6] * requests):
        m.extend(rows, new, 1 << 30)
        pool.extend(None, dev(new), rows=dev(rows))
        m.trim(rows, drop)
        table = pool.page_table.tolist()
        pool.trim(dev(drop), rows=dev(rows))
        assert pool.lens.tolist() == m.lens and pool.counters.tolist() == [len(m.free), 0]
        assert pool.free_pages[:len(m.free)].tolist() == m.free
        assert all(table[q][:m.need(m.lens[q])] == m.table[q][:m.need(m.lens[q])] for q in range(requests))


def test_accepted_drafts_and_ended_requests(pkg):
    pool = pkg.PagePool.empty(requests=4, cols=8, num_pages=32, page_size=16)
    L = 7
    new = dev([L + 1] * 4)
    for lens, accept in (([3, 8, 1, 6], [2, 7, 0, 5]), ([11, 12, 2, 12], [7, 3, 0, 5])):
        pool.extend(None, new)
        pool.trim(accepted=dev(accept), drafts=L)
        assert pool.lens.tolist() == lens
    assert pool.counters.tolist() == [28, 0]
    pool.trim(rows=dev([1, 3]))                      # ended
    assert pool.lens.tolist() == [11, 0, 2, 0] and pool.counters.tolist() == [30, 0]
    pool.trim(batch=4)
    assert pool.lens.tolist() == [0] * 4 and sorted(pool.free_pages.tolist()) == list(range(32))


def test_captured_and_replayed(pkg):
    both, other = Both(pkg, 4, 20, 60, 16), Both(pkg, 4, 20, 60, 16)
    new, drop, rows = dev([9, 9, 9]), dev([4, 0, 9]), dev([3, 1, 0])
    tensors = dict(positions=dev([0] * 27), slots=dev([0] * 27, torch.int64))
    batch = pkg.PagedBatch(dev([0] * 4), dev([0] * 3), dev([[0] * 20] * 3), max_tokens=9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.pool.extend(batch, new, rows=rows, **tensors)
        other.pool.trim(drop, rows=rows)
    for n, d in (([9, 9, 9], [4, 0, 9]), ([1, 0, 9], [0, 5, 1]), ([9, 8, 7], [30, 0, 0])):
        new.copy_(dev(n)), drop.copy_(dev(d))
        graph.replay()
        want = both.extend(n, [3, 1, 0], tokens=27)
        both.trim(d, [3, 1, 0])
        assert batch.tensors[0].tolist() == want[0] and tensors["slots"].tolist()[:sum(n)] == want[4]
        assert other.pool.lens.tolist() == both.m.lens and other.pool.counters.tolist() == both.pool.counters.tolist()
        assert torch.equal(other.pool.page_table[:, :1], both.pool.page_table[:, :1])


def test_no_entries_and_other_streams(pkg):
    pool = pkg.PagePool.empty(requests=2, cols=4, num_pages=8, page_size=16)
    none = dev([]).view(0)
    cu = dev([5])
    pool.extend(pkg.PagedBatch(cu, none, dev([]).view(0, 1), max_tokens=0), none)
    assert cu.tolist() == [0] and pool.counters.tolist() == [8, 0]
    pool.trim(none)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    add = dev([20, 30])
    s.wait_stream(torch.cuda.current_stream())
    pool.extend(None, add, stream=s)
    s.synchronize()
    assert pool.lens.tolist() == [20, 30] and pool.counters.tolist() == [4, 0]


def test_refusals(pkg):
    pool = pkg.PagePool.empty(requests=2, cols=4, num_pages=8, page_size=16)
    add = dev([1, 1])
    with pytest.raises(pkg.DflashError, match="page_size"):
        pkg.PagePool.empty(requests=2, cols=4, num_pages=8, page_size=0).extend(None, add)
    with pytest.raises(pkg.DflashError, match="batch"):
        pool.extend(None, dev([1, 1, 1]))
    with pytest.raises(pkg.DflashError, match="batch"):
        pool.trim(batch=3)
    with pytest.raises(TypeError):
        pool.extend(None, add.long())
    with pytest.raises(ValueError):
        pool.extend(None, add, rows=dev([0]))
    with pytest.raises(ValueError, match="room"):
        pool.extend(None, add, positions=dev([0]), tokens=2)
    with pytest.raises(ValueError):
        pool.trim()
    with pytest.raises(ValueError):
        pool.trim(accepted=add)
    with pytest.raises(ValueError, match="entries"):
        pool.extend(pkg.PagedBatch(dev([0, 0]), dev([0]), dev([[0]]), max_tokens=1), add)
    own = pkg.PagedBatch(dev([0, 0, 0]), pool.lens, pool.page_table, max_tokens=1)
    with pytest.raises(pkg.DflashError, match="rows"):
        pool.extend(own, add, rows=dev([1, 0]))
    assert pool.lens.tolist() == [0, 0]
