"""Books as large as the pages' calls take, and larger ones, which they refuse on the host (CPU only)."""
import ctypes

import pytest

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_pages_refusals import P, book, compact, fork, lib, refused, reserve      # noqa: F401

G = 1 << 40       # addresses that are never read, far enough apart for buffers of 8 GB


def large(**kw):
    return book(**{**dict(table=G, held=2 * G, refs=3 * G, batch=1, max_pages=8, n_pages=100, page=1), **kw})


@pytest.mark.parametrize("kw", [dict(n_pages=2 ** 30 + 1), dict(n_pages=2 ** 31 - 1), dict(max_pages=2 ** 30 + 1), dict(max_pages=2 ** 31 - 1),
                                dict(n_pages=2 ** 31 - 2 ** 20, batch=8192)])
def test_indices_that_could_pass_31_bits(lib, kw):      # noqa: F811
    """A thread looks at up to 2^21 pages (1024 entries of a row) past its last one, in 32 bits."""
    b = large(**kw)
    refused(lib, reserve(lib, b), "2^30")
    refused(lib, fork(lib, b, size=1 << 40), "2^30")
    refused(lib, compact(lib, b, size=1 << 40), "2^30")
    for f in (lib.kvo_paged_fork_workspace, lib.kvo_paged_compact_workspace):
        n = ctypes.c_size_t(7)
        refused(lib, f(b, ctypes.byref(n)), "2^30")
        assert n.value == 0


def test_the_largest_books_are_taken(lib):      # noqa: F811
    for kw in (dict(n_pages=2 ** 30), dict(max_pages=2 ** 30), dict(batch=8192, max_pages=2 ** 18 - 1)):
        for f in (lib.kvo_paged_fork_workspace, lib.kvo_paged_compact_workspace):
            n = ctypes.c_size_t(0)
            assert f(large(**kw), ctypes.byref(n)) == kvo.KVO_OK and n.value > 0
