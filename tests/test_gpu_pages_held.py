"""The pages' bookkeeping where `held` is out of range: clamped, as the header says, and reported."""
import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_gpu_pages import Book, check_moves, i32

pytestmark = pytest.mark.gpu
PAGE = 16


def books(width, batch):
    """Request 0 holds nothing, request 1 all of its row, all others some pages."""
    n = width + 3 * batch + 20
    rows = [[], list(range(3, 3 + width)), [0, 2], [width + 5]] + [[width + 6 + b] for b in range(4, batch)]
    return Book(rows, n, width)


SHAPES = [(6, 4), (300, 7), (1000, 200)]           # tables that one launch takes, and two
BAD = [(-1, None), (-2 ** 31, None), (0, 1), (-7, 5), (0, "most")]


def run(width, batch, low, over):
    book = books(width, batch)
    table, held, refs = book.device()
    raw = held.clone()
    raw[0] = low
    raw[1] = width if over is None else 2 ** 31 - 1 if over == "most" else width + over
    return book, table, raw, refs, i32([0])


@pytest.mark.parametrize("width,batch", SHAPES)
@pytest.mark.parametrize("low,over", BAD)
def test_fork(width, batch, low, over):
    rest = list(range(4, batch))
    size = [len(r) * PAGE for r in books(width, batch).rows]
    for parent, keep in (([-1, -1, 2, 3], [0, 0, 32, 16]),                          # both freed
                         ([0, 1, 2, 3], [0, width * PAGE, 20, 16]),                 # both kept
                         ([0, 1, 1, -1], [0, 16 * width - 16, 16 * width, 0]),      # one cut, and forked from whole
                         ([1, 0, 1, 3], [40, 0, 37, 9]),                            # and from in part; a child of nothing
                         ([2, 3, 0, 1], [32, 16, 0, 5])):
        book, table, held, refs, status = run(width, batch, low, over)
        parent, keep = parent + rest, keep + size[4:]
        moves, _ = book.fork(parent, keep, PAGE)
        got = kvo.paged_fork(table, held, refs, i32(parent), i32(keep), PAGE, status=status)
        book.check(table, held, refs)
        check_moves(got, moves, batch)
        assert int(status.item()) == kvo.DEV_BAD_COUNT
    # more than a parent holds is still refused: the request stays as it is
    book, table, held, refs, status = run(width, batch, low, over)
    got = kvo.paged_fork(table, held, refs, i32([0, 1, 0, 1] + rest), i32([0, 16 * width, 1, 16 * width + 1] + size[4:]), PAGE, status=status)
    book.check(table, held, refs)
    check_moves(got, [], batch)
    assert int(status.item()) == kvo.DEV_BAD_COUNT


@pytest.mark.parametrize("width,batch", SHAPES)
@pytest.mark.parametrize("low,over", BAD)
def test_reserve_and_compact(width, batch, low, over):
    """Reserve gives such a request nothing; compact follows the clamped number; neither touches `held` there."""
    book, table, held, refs, status = run(width, batch, low, over)
    raw = held.clone()
    want = [5 * PAGE if low < 0 else 0, width * PAGE, 3 * PAGE, 4 * PAGE] + [PAGE] * (batch - 4)
    book.reserve([0] + want[1:], PAGE)
    kvo.paged_reserve(table, held, refs, i32(want), PAGE, status=status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    assert torch.equal(held[:2], raw[:2])
    held[:2] = i32([0, width])
    book.check(table, held, refs)
    held[:2] = raw[:2]
    status.zero_()
    for out in (False, True):
        moves = book.compact()
        into = (torch.empty_like(table), torch.empty_like(refs)) if out else ()
        got = kvo.paged_compact(table, held, refs, *into, status=status)
        if out:
            table, refs = into
        check_moves(got, moves, book.n // 2)
        assert int(status.item()) == kvo.DEV_BAD_COUNT and torch.equal(held[:2], raw[:2])
        fixed = held.clone()
        fixed[:2] = i32([0, width])
        book.check(table, fixed, refs)
        # (a hole for the next turn)
        parent, keep = [0, 1, -1] + list(range(3, batch)), [0, width * PAGE, 0] + [len(r) * PAGE for r in book.rows[3:]]
        book.fork(parent, keep, PAGE)
        kvo.paged_fork(table, fixed, refs, i32(parent), i32(keep), PAGE)
        held = fixed.clone()
        held[:2] = raw[:2]
        status.zero_()
