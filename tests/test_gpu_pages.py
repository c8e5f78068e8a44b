"""The pages' bookkeeping (reserve, fork, compact) against the same rules in plain Python, and copies of pages."""
import random

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ceil(a, b):
    return -(-a // b)


class Book:
    """Rows of page ids and the uses of each page; `width` entries to a row."""

    def __init__(self, rows, n_pages, width, pins=()):
        self.rows, self.n, self.width = [list(r) for r in rows], n_pages, width
        self.refs = [0] * n_pages
        for p in [p for r in rows for p in r] + list(pins):
            self.refs[p] += 1

    def device(self):
        table = [r + [-1] * (self.width - len(r)) for r in self.rows]
        return i32(table).view(len(table), self.width), i32([len(r) for r in self.rows]), i32(self.refs)

    def check(self, table, held, refs):
        want = self.device()
        assert torch.equal(held, want[1])
        assert torch.equal(refs, want[2])
        assert torch.equal(table, want[0])

    def free(self):
        return [p for p in range(self.n) if self.refs[p] == 0]

    def reserve(self, want, page):
        free, asked, short = self.free(), 0, False
        for r, w in zip(self.rows, want):
            need = max(0, ceil(w, page) - len(r))
            asked += need
            if need and asked > len(free):
                short = True
            for p in free[asked - need:asked] if asked <= len(free) else []:
                r.append(p)
                self.refs[p] += 1
        return short

    def fork(self, parent, keep, page):
        old = self.rows
        self.rows = [[] if p < 0 else old[p][:ceil(k, page)] for p, k in zip(parent, keep)]
        for r in old:
            for p in r:
                self.refs[p] -= 1
        for r in self.rows:
            for p in r:
                self.refs[p] += 1
        part = [b for b, (r, k) in enumerate(zip(self.rows, keep)) if r and k % page]
        last = {b: self.rows[b][-1] for b in part}
        holders = {}
        for b in part:
            holders.setdefault(last[b], []).append(b)
        copies = [b for b in part if self.refs[last[b]] != len(holders[last[b]]) or b != holders[last[b]][0]]
        free, moves = self.free(), []
        for i, b in enumerate(copies):
            self.refs[last[b]] -= 1
            self.rows[b].pop()
            if i < len(free):
                self.rows[b].append(free[i])
                self.refs[free[i]] = 1
                moves.append((last[b], free[i]))
        return moves, len(copies) > len(free)

    def compact(self):
        live = sum(x > 0 for x in self.refs)
        moves = list(zip([p for p in range(live, self.n) if self.refs[p]], [p for p in range(live) if not self.refs[p]]))
        to = dict(moves)
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves


def check_moves(got, moves, size):
    src, dst, count = got
    assert int(count.item()) == len(moves)
    assert src.tolist() == [a for a, _ in moves] + [-1] * (size - len(moves))
    assert dst.tolist() == [b for _, b in moves] + [-1] * (size - len(moves))


@pytest.mark.parametrize("batch,n_pages,page,most,seed", [
    (1, 1, 16, 1, 0), (1, 5, 16, 3, 1), (3, 17, 16, 9, 2), (7, 63, 32, 8, 3), (33, 1000, 64, 40, 4), (130, 4096, 128, 33, 5),
    (64, 4097, 16, 90, 6), (64, 8191, 16, 90, 7), (300, 40003, 16, 120, 8), (1030, 9000, 16, 7, 9), (256, 300000, 16, 1000, 10),
    (4000, 20000, 32, 4, 11), (8192, 33000, 16, 3, 12), (256, 700001, 16, 1200, 13)])
def test_a_long_run_matches_plain_python(batch, n_pages, page, most, seed):
    """Forks, cuts, reorders, frees, reservations and compactions in turn, the pool often short of pages."""
    rng = random.Random(seed)
    pins = rng.sample(range(n_pages), min(n_pages // 20, 50))
    book = Book([[] for _ in range(batch)], n_pages, most, pins)
    table, held, refs = book.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = [0] * batch
    short = 0
    for step in range(6 if batch * most < 100000 else 3):
        want = [rng.choice([0, rng.randint(0, most * page)]) if rng.random() < 0.7 else lens[b] for b in range(batch)]
        lack = book.reserve(want, page)
        kvo.paged_reserve(table, held, refs, i32(want), page, status=status)
        book.check(table, held, refs)
        assert int(status.item()) == (kvo.DEV_NO_PAGES if lack else 0)
        status.zero_()
        lens = [min(len(r) * page, max(w, 0)) for r, w in zip(book.rows, want)]
        parent = [rng.choice([b, b, -1, rng.randrange(batch)]) for b in range(batch)]
        top = [0 if p < 0 else len(book.rows[p]) * page for p in parent]
        keep = [rng.choice([t, rng.randint(0, t), min(t, lens[p])]) for t, p in zip(top, parent)]
        moves, lack = book.fork(parent, keep, page)
        got = kvo.paged_fork(table, held, refs, i32(parent), i32(keep), page, status=status)
        book.check(table, held, refs)
        check_moves(got, moves, batch)
        assert int(status.item()) == (kvo.DEV_NO_PAGES if lack else 0)
        status.zero_()
        short += lack
        lens = [min(k, len(r) * page) for k, r in zip(keep, book.rows)]
        before = (table.clone(), refs.clone())
        moves = book.compact()
        if step % 2:
            got = kvo.paged_compact(table, held, refs, status=status)
        else:
            out = (torch.empty_like(table), torch.empty_like(refs))
            got = kvo.paged_compact(table, held, refs, *out, status=status)
            assert torch.equal(table, before[0]) and torch.equal(refs, before[1])
            table, refs = out
        book.check(table, held, refs)
        check_moves(got, moves, n_pages // 2)
        assert int(status.item()) == 0


def test_a_shared_part_filled_page_goes_to_the_lowest_that_holds_it_so():
    page = 16
    book = Book([[3, 4], [], [], [], []], 9, 4)
    table, held, refs = book.device()
    got = kvo.paged_fork(table, held, refs, i32([-1, 0, 0, 0, 0]), i32([0, 20, 32, 20, 17]), page)
    # request 2 holds page 4 in full: nobody else may write into it
    check_moves(got, [(4, 0), (4, 1), (4, 2)], 5)
    assert table.tolist() == [[-1] * 4, [3, 0, -1, -1], [3, 4, -1, -1], [3, 1, -1, -1], [3, 2, -1, -1]]
    assert held.tolist() == [0, 2, 2, 2, 2] and refs.tolist() == [1, 1, 1, 4, 1, 0, 0, 0, 0]
    # without that one the lowest keeps the page; a kept prefix (a use of the caller's own) keeps it from all
    book = Book([[3, 4], [], []], 9, 4)
    table, held, refs = book.device()
    check_moves(kvo.paged_fork(table, held, refs, i32([-1, 0, 0]), i32([9, 20, 20]), page), [(4, 0)], 3)
    assert table[1:, :2].tolist() == [[3, 4], [3, 0]]
    book = Book([[3, 4], [], []], 9, 4, pins=[4])
    table, held, refs = book.device()
    check_moves(kvo.paged_fork(table, held, refs, i32([-1, 0, 0]), i32([9, 20, 20]), page), [(4, 0), (4, 1)], 3)
    assert refs.tolist() == [1, 1, 0, 2, 1, 0, 0, 0, 0]


def test_what_is_out_of_range_is_reported_and_left_alone():
    page = 16
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for parent, keep in (([5, 1], [16, 16]), ([-2, 1], [16, 16]), ([0, 1], [-1, 16]), ([0, 1], [33, 16]), ([1, 1], [17, 16])):
        book = Book([[1, 2], [5]], 12, 3)
        table, held, refs = book.device()
        check_moves(kvo.paged_fork(table, held, refs, i32(parent), i32(keep), page, status=status), [], 2)
        book.check(table, held, refs)
        assert int(status.item()) == kvo.DEV_BAD_COUNT
        status.zero_()
    for want in ([-1, 40], [49, 40], [2 ** 31 - 1, 40]):
        book = Book([[1, 2], [5]], 12, 3)
        table, held, refs = book.device()
        kvo.paged_reserve(table, held, refs, i32(want), page, status=status)
        book.reserve([0, 40], page)
        book.check(table, held, refs)
        assert int(status.item()) == kvo.DEV_BAD_COUNT
        status.zero_()
    # page ids outside the pool: not followed
    table, held, refs = i32([[1, 99], [-7, 2]]), i32([2, 2]), i32([0, 1, 1, 0])
    got = kvo.paged_compact(table, held, refs, status=status)
    check_moves(got, [(2, 0)], 2)
    assert table.tolist() == [[1, 99], [-7, 0]] and refs.tolist() == [1, 1, 0, 0]
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    status.zero_()
    kvo.paged_fork(table, held, refs, i32([1, -1]), i32([32, 0]), page, status=status)
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    assert table.tolist() == [[-7, 0], [-1, -1]] and refs.tolist() == [1, 0, 0, 0]


def test_no_requests_and_a_pool_of_one_page():
    table, held, refs = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), i32([]), i32([0, 1, 0])
    kvo.paged_reserve(table, held, refs, i32([]), 16)
    src, dst, count = kvo.paged_fork(table, held, refs, i32([]), i32([]), 16, count=i32([7]))
    assert src.numel() == 0 and int(count.item()) == 0
    src, dst, count = kvo.paged_compact(table, held, refs)
    assert (src.tolist(), dst.tolist(), count.tolist(), refs.tolist()) == ([1], [0], [1], [1, 0, 0])
    src, dst, count = kvo.paged_compact(table, held, i32([1]))
    assert src.numel() == 0 and int(count.item()) == 0


def test_calls_into_given_buffers_and_graphs():
    """A captured step (cut, reserve, compact) replayed on changing lengths, with buffers that hold anything before."""
    page, batch, width, n_pages = 32, 40, 60, 5000
    rng = random.Random(5)
    book = Book([[] for _ in range(batch)], n_pages, width)
    book.reserve([rng.randint(0, 1500) for _ in range(batch)], page)
    table, held, refs = book.device()
    keep, want = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    parent = i32(list(range(batch)))
    src, dst, count = i32([9] * batch), i32([9] * batch), i32([9])
    csrc, cdst, ccount = i32([9] * (n_pages // 2)), i32([9] * (n_pages // 2)), i32([9])
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    ws2 = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")

    def step():
        kvo.paged_fork(table, held, refs, parent, keep, page, src, dst, count, ws)
        kvo.paged_reserve(table, held, refs, want, page)
        kvo.paged_compact(table, held, refs, None, None, csrc, cdst, ccount, ws2)

    lens = [len(r) * page for r in book.rows]

    def host():
        for b in range(batch):
            lens[b] = rng.randint(0, min(lens[b], len(book.rows[b]) * page))
        keep.copy_(i32(lens))
        moves, _ = book.fork(list(range(batch)), lens, page)
        w = [min(x + rng.randint(0, 200), width * page) for x in lens]
        want.copy_(i32(w))
        book.reserve(w, page)
        for b in range(batch):
            lens[b] = w[b]
        return moves, book.compact()

    def look(moves):
        torch.cuda.synchronize()
        check_moves((src, dst, count), moves[0], batch)
        check_moves((csrc, cdst, ccount), moves[1], n_pages // 2)
        book.check(table, held, refs)

    moves = host()
    step()
    look(moves)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(4):
        moves = host()
        ws.fill_(rng.randrange(256))
        graph.replay()
        look(moves)


def pools(layers, n_pages, hkv, page, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = ((layers,) if layers else ()) + (n_pages, hkv, page, d)
    raw = lambda: torch.randint(0, 256, shape if dtype == E4M3 else shape[:-1] + (2 * d,), generator=g, device="cuda", dtype=torch.uint8)
    k, v = raw().view(dtype), raw().view(dtype)
    scales = [torch.rand(shape[:-2], generator=g, device="cuda") for _ in range(2)] if dtype == E4M3 else [None, None]
    return k, v, *scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("layers,n_pages,hkv,page,d,moves", [
    (0, 9, 1, 16, 64, 2), (1, 2, 1, 16, 64, 1), (3, 40, 2, 32, 128, 13), (2, 64, 8, 64, 128, 30), (0, 31, 3, 128, 128, 15),
    (5, 700, 5, 16, 64, 345), (0, 20, 16, 128, 128, 9)])
def test_copies_are_exact(dtype, layers, n_pages, hkv, page, d, moves):
    k, v, ks, vs = pools(layers, n_pages, hkv, page, d, dtype, n_pages)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(moves)).tolist()
    src, dst = i32(order[:moves] + [-1]), i32(order[moves:2 * moves] + [-1])
    for count in (None, moves, moves // 2, 0):
        want = []
        n = moves if count is None else count
        for x in (k, v, ks, vs):
            if x is None:
                continue
            y = x.view(torch.uint8).clone() if x.dtype == E4M3 else x.view(torch.int16).clone() if x.dtype == torch.bfloat16 else x.clone()
            at = y if layers else y[None]
            at[:, dst[:n].long()] = at[:, src[:n].long()]
            want.append((x, y))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvo.paged_copy(k, v, src[:moves] if count is None else src, dst[:moves] if count is None else dst,
                       None if count is None else i32([count]), k_scale=ks, v_scale=vs, status=status)
        for x, y in want:
            assert torch.equal(x.view(y.dtype), y)
        assert int(status.item()) == 0


def test_copy_skips_what_is_out_of_range():
    k, v, _, _ = pools(0, 8, 2, 16, 64, torch.bfloat16, 1)
    want = k.view(torch.int16).clone()
    want[5] = want[1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvo.paged_copy(k, v, i32([1, 8, -1, 2, 3, 4]), i32([5, 6, 6, 8, -5, 4]), status=status)
    assert torch.equal(k.view(torch.int16), want) and int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    status.zero_()
    kvo.paged_copy(k, v, i32([1]), i32([5]), i32([2]), status=status)
    assert torch.equal(k.view(torch.int16), want) and int(status.item()) == kvo.DEV_BAD_COUNT
    status.zero_()
    kvo.paged_copy(k, v, i32([2]), i32([6]), i32([-3]), status=status)
    assert torch.equal(k.view(torch.int16), want) and int(status.item()) == kvo.DEV_BAD_COUNT


def test_copy_past_four_gigabytes():
    """A pool of 4.5 GB a side: offsets pass 32 bits within a layer and between layers."""
    k = torch.empty(3, 11000, 8, 64, 128, dtype=E4M3, device="cuda").view(torch.uint8)
    v = torch.empty_like(k)
    k[1, 10990], v[2, 10999] = 17, 23
    k[2, 10990], v[1, 10999] = 18, 24
    s = torch.ones(3, 11000, 8, device="cuda")
    s[2, 10990] = 4.0
    kvo.paged_copy(k.view(E4M3), v.view(E4M3), i32([10990, 10999]), i32([3, 10997]), k_scale=s, v_scale=s.clone())
    assert (k[1, 3] == 17).all() and (k[2, 3] == 18).all() and (v[2, 10997] == 23).all() and (v[1, 10997] == 24).all()
    assert (s[2, 3] == 4.0).all()
