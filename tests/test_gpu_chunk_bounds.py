"""Attention of new tokens over a paged cache under bounds of any size, and next to requests whose offsets are bad."""
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


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bounds", [{}, dict(max_new=6), dict(max_new=6, max_len=300000)])
@pytest.mark.parametrize("batch", [5, 40])
@pytest.mark.parametrize("spoil", [{2: 13}, {2: 9, 3: 7}, {1: 8, 2: 10}, {1: 0}, {2: 11, 4: 19}])
def test_neighbours_of_a_bad_offset(spoil, batch, bounds, e4m3):
    """One offset stands between two requests: the one that is still served gets all of its rows, with its new number of tokens."""
    c = Case(batch, 64, 1, 2, 16, e4m3, [6] * batch, [60] * batch)
    cu = list(c.cu)
    for i, x in spoil.items():
        cu[i] = x
    total, end, rows = c.cu[-1], 0, {}
    for b in range(batch):
        if 0 <= cu[b] <= cu[b + 1] <= total:
            if cu[b] >= end and not (bounds and cu[b + 1] - cu[b] > 8):      # (more new tokens than 16 rows: left out)
                rows[b] = (cu[b], cu[b + 1])
            end = max(end, cu[b + 1])
    assert any(rows[b] != (c.cu[b], c.cu[b + 1]) for b in rows)
    o, lse = (torch.full(s, 3.0, dtype=t, device="cuda") for s, t in ((c.q.shape, torch.bfloat16), (c.q.shape[:2], torch.float32)))
    status = i32([0])
    kvo.paged_chunk_attn(c.q, c.kp, c.vp, c.table, i32(c.lens), i32(cu), k_scale=c.scales[0], v_scale=c.scales[1], o=o, lse=lse, status=status, **bounds)
    assert int(status.item()) == (0 if len(rows) == batch else kvo.DEV_BAD_COUNT)
    served = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, e in rows.values():
        served[a:e] = True
    assert (o[~served] == 3.0).all() and (lse[~served] == 3.0).all()
    assert (o[served] != 3.0).any(-1).all()
    c.new, c.cu = [rows[b][1] - rows[b][0] if b in rows else 0 for b in range(batch)], [rows[b][0] if b in rows else 0 for b in range(batch)]
    c.check(o, lse, requests=sorted(rows)[:6] + sorted(rows)[-2:])


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [-1, -2, -2 ** 31, -2 ** 31 + 1, "n_pages", 2 ** 31 - 1, 2 ** 30])
def test_page_ids_of_any_value(bad, e4m3, few):
    """Whatever an entry holds that names no page, its tokens add nothing."""
    new, lens = ([4, 3, 1], [300, 30, 9]) if few else ([70, 3, 1], [300, 30, 9])
    c = Case(61, 64, 2, 4, 16, e4m3, new, lens)
    bad = c.n_pages if bad == "n_pages" else bad
    c.table[0, 3], c.table[0, 17], c.table[1, 0], c.table[2, 0] = bad, bad, bad, bad
    status = i32([0])
    o, lse = c.call(status=status, max_new=4 if few else 0)
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    c.check(o, lse, rows=[0, 1, 2, 33, -1], heads=[0, 7], hide={(0, 3), (0, 17), (1, 0), (2, 0)})
    assert (o[sum(new) - 1] == 0).all() and (lse[sum(new) - 1] == -float("inf")).all()
