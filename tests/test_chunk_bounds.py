"""Bounds of any size in attention of new tokens over a paged cache: which kernels a call takes shows in its workspace (CPU only)."""
import pytest

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_chunk_refusals import cache, lib, refused, size      # noqa: F401

BIG = [2 ** 63 - 1, 2 ** 62, 2 ** 61 + 1, 2 ** 60, 2 ** 59 + 3, 2 ** 32, 2 ** 31]


@pytest.mark.parametrize("r", range(1, 17))
@pytest.mark.parametrize("fmt", [0, 1])
def test_large_bounds_are_bounds(lib, r, fmt):      # noqa: F811
    """An upper bound beyond 16 rows says as much as none: the workspace of long chunks, which a call with less refuses."""
    c = cache(fmt=fmt, n_pages=10 ** 5, max_pages=10 ** 4)
    want = size(lib, c, hq=2 * r, total=1000)
    assert want[0] == kvo.KVO_OK
    for max_new in BIG + [16 // r + 1]:
        assert size(lib, c, hq=2 * r, total=1000, max_new=max_new) == want
    few = size(lib, c, hq=2 * r, total=1000, max_new=16 // r)
    assert few[0] == kvo.KVO_OK and few != want
    for max_len in BIG:
        assert size(lib, c, hq=2 * r, total=1000, max_new=16 // r, max_len=max_len) == few
