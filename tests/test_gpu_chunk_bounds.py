"""Attention of new tokens over a paged cache under bounds of any size."""
import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_gpu_chunk import Case, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("r", [1, 2, 3, 4, 8, 16])
def test_a_bound_beyond_all_is_none(e4m3, r):
    """max_new and max_len are upper bounds: the largest numbers leave no request out and change no bit."""
    c = Case(r, 64, 2, r, 32, e4m3, [40, 1, 9], [300, 20, 9])
    status = i32([0])
    want = c.call(status=status)
    for bound in (2 ** 63 - 1, 2 ** 62, 2 ** 60, 2 ** 31):
        o, lse = (torch.full(s, 3.0, dtype=t, device="cuda") for s, t in ((c.q.shape, torch.bfloat16), (c.q.shape[:2], torch.float32)))
        c.call(o=o, lse=lse, status=status, max_new=bound, max_len=bound)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert int(status.item()) == 0
    c.check(*want, rows=[0, 3, 17, -1], heads=[0, 2 * r - 1])
