"""Forks of many requests over long rows, which two launches make: part-filled pages shared by many, again and again."""
import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_gpu_pages import Book, check_moves, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,width,parents,n_pages", [(8192, 20, 2000, 60000), (8192, 20, 1, 60000), (5000, 40, 700, 4096), (300, 500, 100, 3000)])
def test_many_forks_of_part_filled_pages(batch, width, parents, n_pages):
    """Every request becomes a copy of one of some, whose last page is filled in part: the lowest keeps it, all others get a page."""
    page = 16
    rows = [[p, n_pages - 1 - p] for p in range(parents)] + [[] for _ in range(batch - parents)]
    want = Book(rows, n_pages, width)
    state = want.device()
    parent = [(b * 7) % parents for b in range(batch)]
    keep = [17 + b % 15 for b in range(batch)]
    moves, lack = want.fork(parent, keep, page)
    args = i32(parent), i32(keep)
    outs = []
    for _ in range(40):
        status = i32([0])
        book = [x.clone() for x in state]
        got = kvo.paged_fork(*book, *args, page, status=status)
        outs.append((book, got, status))
    for book, got, status in outs:
        want.check(*book)
        assert int(status.item()) == (kvo.DEV_NO_PAGES if lack else 0)
    check_moves(outs[0][1], moves, batch)
    for _, got, _ in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got, outs[0][1]))
