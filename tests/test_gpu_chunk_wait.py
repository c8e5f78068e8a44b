"""The bounded waits of attention of new tokens over a paged cache, made to run out.

The test switch (kvo_set_call_wait_test) makes the kernels announce one load without copying it, so that the wait for it
never completes: it gives up after the limit, sets KVO_DEV_TIMEOUT in the caller's status word and the call returns, with
every copy that it did issue landed.  The same call afterwards, with the switch off, gives the bits that it gave before.
Nothing faults or hangs: the only missing piece is a copy that is never issued."""
import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_gpu_call_wait import gen, i32, normal, paged, runs_out

pytestmark = pytest.mark.gpu


def run_out(new, lens, hkv, r, d, page, e4m3, tile, fill, **kw):
    g = gen(tile)
    a, scales = paged(g, lens, hkv, r, d, page, e4m3, max(-(-n // page) for n in lens) + 1)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = normal(g, cu[-1], hkv * r, d)
    ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
    call = lambda status: kvo.paged_chunk_attn(q, *a[1:], i32(cu), workspace=ws, status=status, **scales, **kw)
    status = i32([0])
    want = call(status)
    assert int(status.item()) == 0
    ws.fill_(fill)
    runs_out(call, tile)
    status = i32([0])
    got = call(status)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(status.item()) == 0


@pytest.mark.parametrize("fill", [0x7F, 0xFF])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [0, 1, 2, 3, 6, 9])        # K of the range's tile i is 2 i, V is 2 i + 1
def test_long_chunks(e4m3, d, tile, fill):
    """Two tiles of rows, one, and single tokens; ranges that end inside a request."""
    run_out([300, 1, 40, 1], [2000, 700, 1100, 1300], 2, 4, d, 64, e4m3, tile, fill)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tile", [0, 1])
def test_one_tile_of_rows(e4m3, tile):
    run_out([20], [6000], 1, 4, 128, 32, e4m3, tile, 0x7F)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("max_len", [0, 3000])
def test_few_new_tokens(e4m3, tile, max_len):
    run_out([4, 1, 3, 2], [2900, 700, 1100, 64], 2, 4, 128, 32, e4m3, tile, 0x7F, max_new=4, max_len=max_len)
