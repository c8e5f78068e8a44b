"""The bounded waits of the context-free attention calls, made to run out.

The test switch (kvo_set_call_wait_test) makes the kernels announce one tile without copying it, so the wait for it can
never complete.  The wait must give up after the limit, set KVO_DEV_TIMEOUT in the caller's status word and let the call
return, with every copy it did issue landed; the same call afterwards, with the switch off, gives the bits that it gave
before.  Nothing faults or hangs: the only missing piece is a copy that is never issued."""
import contextlib
import time

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g).bfloat16().cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@contextlib.contextmanager
def skipped(tile, limit_ns=20_000_000):
    kvo.set_call_wait_test(limit_ns, tile)
    try:
        yield
    finally:
        kvo.set_call_wait_test()


def runs_out(call, tile):
    """The call with a tile left out: in time, and the status bit."""
    status = i32([0])
    with skipped(tile):
        t0 = time.perf_counter()
        call(status)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5.0                  # the limit, not a hang
    assert int(status.item()) == kvo.DEV_TIMEOUT


def paged(g, lens, hkv, r, d, page, e4m3, cap):
    """A call's arguments: its own pages for each request, of which a table of `cap` entries names those it needs."""
    need = [(n + page - 1) // page for n in lens]
    n_pages = sum(need) + 1
    table = torch.zeros(len(lens), cap, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(at, at + n)
        at += n
    kp, vp = (torch.randn(n_pages, hkv, page, d, generator=g).to(E4M3 if e4m3 else torch.bfloat16).cuda() for _ in range(2))
    ks, vs = (torch.full((n_pages, hkv), 0.5, device="cuda") if e4m3 else None for _ in range(2))
    return (normal(g, len(lens), hkv * r, d), kp, vp, table.cuda(), i32(lens)), dict(k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("fill", [0x7F, 0xFF, 0x01])
@pytest.mark.parametrize("e4m3,tile", [(True, 0), (True, 1), (False, 3), (False, 1)])
def test_ranges_after_a_wait_that_ran_out(e4m3, tile, fill):
    """Warps that stop leave groups of their range without an entry in the workspace; the join must not take what lies
    there for one, whatever it is."""
    a, kw = paged(gen(tile), [(13 * i) % 200 for i in range(400)], 8, 2, 64, 16, e4m3, 13)
    ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
    want = kvo.paged_attn(*a, workspace=ws, **kw)
    ws.fill_(fill)
    runs_out(lambda status: kvo.paged_attn(*a, workspace=ws, status=status, **kw), tile)
    status = i32([0])
    got = kvo.paged_attn(*a, workspace=ws, status=status, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(status.item()) == 0


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("lens,cap,tile", [([3000, 0, 700, 5000], 7000, 0), ([3000, 0, 700, 5000], 7000, 1),     # ranges
                                           ([900, 70], 60, 0), ([5], 60, 0), ([4000, 3001], 320, 1)])            # clusters
def test_paged_attention_wait_runs_out(e4m3, lens, cap, tile):
    a, kw = paged(gen(len(lens)), lens, 2, 4, 128, 16, e4m3, cap)
    want = kvo.paged_attn(*a, **kw)
    runs_out(lambda status: kvo.paged_attn(*a, status=status, **kw), tile)
    got = kvo.paged_attn(*a, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# n tiles of 128 keys: loads 0 .. 2n - 1; the last V goes through a barrier of its own where it is cut
@pytest.mark.parametrize("d,hkv,r,nq,nk,loads", [
    (128, 1, 4, [130], None, [0, 1, 2, 3]),                      # two tiles, the last one cut: nothing but the first loads
    (64, 2, 4, [3, 0, 129, 1, 256], None, [0, 1, 3]),            # short prompts in one call, whole and cut tiles
    (128, 8, 4, [1300], None, [0, 7, 16, 21]),                   # loads that wait for a stage of the ring
    (128, 1, 4, [5], [1500], [0, 1, 2, 3]),                      # split over clusters: parts of one to a few tiles
    (64, 1, 2, [40, 3], [3000, 17], [0, 1, 4]),
    (128, 8, 4, [200], [6000], [0, 5, 14])])
def test_prompt_attention_wait_runs_out(d, hkv, r, nq, nk, loads):
    g = gen(d + r)
    cuts = lambda counts: [sum(counts[:i]) for i in range(len(counts) + 1)]
    cq, ck = cuts(nq), cuts(nk or nq)
    q, k, v = normal(g, cq[-1], hkv * r, d), normal(g, ck[-1], hkv, d), normal(g, ck[-1], hkv, d)
    call = lambda status=None: kvo.prompt_attn(q, k, v, i32(cq), i32(ck), status=status)
    want = call()
    for load in loads:
        runs_out(call, load)
        status = i32([0])
        got = call(status)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(status.item()) == 0
