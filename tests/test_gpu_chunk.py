"""Attention of new tokens over a paged cache against a plain 64-bit reference."""
import math
import random

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cuts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


class Case:
    """Pools with NaN wherever no request's token lies, a shuffled table, and the keys and values in 64 bits."""

    def __init__(self, seed, d, hkv, r, page, e4m3, new, lens, q_scale=1.0, k_scale=1.0, spare=0, wild=False):
        g = torch.Generator().manual_seed(seed)
        self.d, self.hkv, self.r, self.page, self.e4m3, self.new, self.lens = d, hkv, r, page, e4m3, new, lens
        need = [-(-n // page) for n in lens]
        self.n_pages, width = sum(need) + 3, max(need + [1]) + 1
        order = torch.randperm(self.n_pages, generator=g).tolist()
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        dtype = E4M3 if e4m3 else torch.bfloat16
        pools, self.scales, self.rows = [], [], []
        for name in "kv":
            pool = torch.full((self.n_pages, hkv, page, d), math.nan).to(dtype)
            scale = torch.ones(self.n_pages, hkv)
            if e4m3:
                scale = torch.exp2(torch.randint(-9, -6, scale.shape, generator=g).float()) * (0.75 + 0.5 * torch.rand(scale.shape, generator=g))
                if wild:
                    scale = scale * torch.exp2(torch.randint(-40, 30, scale.shape, generator=g).float()) if name == "v" else scale
            at, rows = 0, []
            for b, n in enumerate(lens):
                mine = order[at:at + need[b]]
                at += need[b]
                table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
                x = torch.randn(need[b] * page, hkv, d, generator=g) * (k_scale if name == "k" else 1.0) * (100.0 if e4m3 else 1.0)
                x = x.clamp(-448, 448).to(dtype)
                y = x.view(need[b], page, hkv, d).transpose(1, 2).contiguous()
                for i, p in enumerate(mine):
                    m = min(page, n - i * page)
                    pool[p, :, :m] = y[i, :, :m]
                full = x.double()[:n]
                if e4m3 and n:
                    full = full * torch.stack([scale[mine[t // page]] for t in range(n)]).double()[..., None]
                rows.append(full)
            pools.append(pool.cuda())
            self.scales.append(scale.cuda() if e4m3 else None)
            self.rows.append(rows)
        self.kp, self.vp, self.table = *pools, table.cuda()
        self.cu = cuts(new)
        self.q = (torch.randn(self.cu[-1] + spare, hkv * r, d, generator=g) * q_scale).bfloat16().cuda()

    def call(self, q=None, **kw):
        kw = {**dict(k_scale=self.scales[0], v_scale=self.scales[1]), **kw}
        return kvo.paged_chunk_attn(self.q if q is None else q, self.kp, self.vp, self.table, i32(self.lens), i32(self.cu), **kw)

    def check(self, o, lse, rows=None, heads=None, requests=None, hide=()):
        """Rows (token, head), each against the attention of its own request; `hide`: (request, page) to leave out."""
        for b in range(len(self.new)) if requests is None else requests:
            n, have = self.new[b], self.lens[b]
            for i in range(n) if rows is None else sorted({x % n for x in rows if n}):
                see = max(have - n + i + 1, 0)
                keep = [t for t in range(see) if (b, t // self.page) not in hide]
                for h in range(self.hkv * self.r) if heads is None else heads:
                    q, g = self.q[self.cu[b] + i, h].double().cpu(), h // self.r
                    k, v = self.rows[0][b][:see, g], self.rows[1][b][:see, g]
                    if hide:
                        k, v = k[keep], v[keep]
                    # weights are rounded to bf16, next to e4m3 pages to f16 with the page's v_scale in them (its logarithm in
                    # fp32, and steps of 2^-24 for small ones): twice bf16's half step covers both
                    want, wl, tol, tl = ref.attention(q, k, v, 2 * ref.BF16 if self.e4m3 else ref.BF16)
                    if self.e4m3 and len(keep):
                        # q as two e4m3 values: each within 2^-17 of the row's largest
                        ds = float(2.0 ** -17 * q.abs().max() * k.abs().sum(1).max() / math.sqrt(self.d))
                        tol = tol + 2 * ds * (torch.softmax(k @ q / math.sqrt(self.d), 0) @ v.abs())
                        tl += ds
                    ref.check(o[self.cu[b] + i, h], want, tol, f"o of request {b}, token {i}, head {h}")
                    got = float(lse[self.cu[b] + i, h])
                    assert got == wl or abs(got - wl) <= tl, (b, i, h, got, wl)


SHAPES = [
    # d, hkv, r, page, new, lens
    (128, 1, 1, 16, [1], [1]), (64, 1, 1, 128, [1], [1]), (128, 1, 4, 32, [4], [130]), (64, 2, 4, 16, [3, 0, 129, 1, 64], [3, 5, 300, 1, 64]),
    (128, 2, 1, 64, [257], [257]), (64, 1, 16, 128, [40, 9], [140, 9]), (128, 1, 3, 16, [50, 200], [50, 333]), (128, 1, 7, 64, [91], [1000]),
    (64, 1, 12, 32, [33, 1], [33, 700]), (128, 2, 2, 128, [5, 1, 70], [300, 128, 70]), (128, 1, 8, 16, [1, 1, 1], [500, 1, 255]),
    (128, 8, 4, 64, [2, 5, 1, 3], [900, 70, 2100, 3]), (64, 2, 5, 64, [20, 30, 4], [20, 1029, 4]), (128, 1, 16, 32, [17], [1500])]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,hkv,r,page,new,lens", SHAPES)
def test_chunks_match_reference(e4m3, d, hkv, r, page, new, lens):
    c = Case(sum(lens) + r, d, hkv, r, page, e4m3, new, lens, q_scale=1.5)
    status = i32([0])
    o, lse = c.call(status=status)
    assert int(status.item()) == 0
    which = dict(rows=None if sum(new) * hkv * r < 400 else [0, 1, 2, 4, 31, 32, 63, 64, 85, 127, 128, 199, -1],
                 heads=None if hkv * r <= 8 else [0, r - 1, hkv * r - 1])
    c.check(o, lse, **which)
    again = c.call(max_new=max(new), max_len=max(lens))        # up to 16 rows: other kernels
    if max(new) * r > 16:
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    else:
        c.check(*again, **which)
        third = c.call(max_new=max(new), max_len=max(lens))
        assert torch.equal(again[0], third[0]) and torch.equal(again[1], third[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cap", [0, 100000])                  # clusters, ranges and their join
@pytest.mark.parametrize("d,hkv,r,page,new,lens", [
    (128, 2, 4, 16, [4, 0, 1, 3, 2], [2000, 5, 1, 700, 128]), (64, 1, 1, 32, [16, 5, 16], [16, 400, 1030]), (128, 8, 2, 64, [1, 4], [3001, 2500]),
    (64, 4, 16, 128, [1, 1, 0, 1], [900, 3, 7, 128]), (128, 1, 3, 32, [5, 2, 5], [5, 3, 611]), (64, 2, 8, 16, [2, 1], [1000, 66]),
    (128, 1, 8, 128, [1], [5000]), (128, 4, 5, 16, [3] * 40, [40 * i + 3 for i in range(40)]), (64, 1, 4, 16, [4] * 300, [7 * i % 90 + 4 for i in range(300)])])
def test_few_new_tokens(e4m3, cap, d, hkv, r, page, new, lens):
    """Up to 16 rows to a request, each with its own last key."""
    c = Case(sum(lens), d, hkv, r, page, e4m3, new, lens, q_scale=2.0, spare=3)
    status = i32([0])
    o, lse = (torch.full(s, 3.0, dtype=t, device="cuda") for s, t in ((c.q.shape, torch.bfloat16), (c.q.shape[:2], torch.float32)))
    c.call(o=o, lse=lse, status=status, max_new=max(new), max_len=max(cap, max(lens)))
    assert int(status.item()) == 0
    some = None if len(new) < 10 else range(0, len(new), len(new) // 12)
    c.check(o, lse, heads=None if hkv * r <= 8 else [0, r - 1, hkv * r - 1], requests=some)
    assert (o[c.cu[-1]:] == 3.0).all() and (lse[c.cu[-1]:] == 3.0).all()
    assert (o[:c.cu[-1]] != 3.0).any(-1).all()
    again = c.call(max_new=max(new), max_len=max(cap, max(lens)))
    assert torch.equal(again[0][:c.cu[-1]], o[:c.cu[-1]]) and torch.equal(again[1][:c.cu[-1]], lse[:c.cu[-1]])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cap", [0, 200000])
def test_few_new_tokens_out_of_range(e4m3, cap):
    """Rows that see nothing, more new tokens than announced, pages that do not exist, NaN in a neighbour's pages."""
    c = Case(41, 64, 2, 4, 16, e4m3, [4, 3, 4, 2], [2, 0, 300, 80])
    status = i32([0])
    kw = dict(max_new=4, max_len=max(cap, 300))
    o, lse = c.call(status=status, **kw)
    assert int(status.item()) == 0
    c.check(o, lse)
    for p in c.table[2, :19].tolist():
        c.kp.view(torch.uint8)[p], c.vp.view(torch.uint8)[p] = 255, 255
    o2, lse2 = c.call(**kw)
    assert o2[7:11].isnan().all() and torch.equal(o2[:7], o[:7]) and torch.equal(o2[11:], o[11:])
    c = Case(43, 64, 2, 4, 16, e4m3, [4, 3, 4, 2], [100, 50, 300, 80])
    c.table[2, 3], c.table[0, 6], c.table[3, 0] = -1, c.n_pages, 2 ** 31 - 1
    o, lse = c.call(status=status, **kw)
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    c.check(o, lse, hide={(2, 3), (0, 6), (3, 0)})
    c = Case(47, 64, 2, 4, 16, e4m3, [4, 30, 4, 2], [100, 50, 300, 80])
    status.zero_()
    o = torch.full(c.q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    c.call(o=o, status=status, **kw)
    assert int(status.item()) == kvo.DEV_BAD_COUNT and (o[4:34] == 3.0).all()
    o, lse = c.call(o=o, **kw)
    c.check(o, lse, requests=[0, 2, 3])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,hkv,r,page,new,lens,q_scale", [
    (128, 8, 4, 64, [500], [9001], 1.0), (128, 2, 4, 16, [700, 1, 33], [5000, 4001, 1033], 6.0), (64, 4, 8, 32, [300, 5], [2100, 8000], 3.0),
    (128, 1, 1, 128, [2500], [2500], 20.0), (64, 8, 2, 64, [1300], [1300], 1.0)])
def test_long_chunks(e4m3, d, hkv, r, page, new, lens, q_scale):
    """Items that range borders cut, and scores that spread far enough for the running maximum to rise late."""
    c = Case(sum(lens), d, hkv, r, page, e4m3, new, lens, q_scale=q_scale)
    o, lse = c.call()
    c.check(o, lse, rows=[0, 1, 31, 32, 127, 255, 256, 299, 640, -1], heads=[0, hkv * r - 1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_requests_of_all_kinds(e4m3):
    """Single tokens, pieces and empty requests side by side: one tile of rows or two, in every order, many items to a CTA."""
    rng = random.Random(3)
    new = [rng.choice([0, 1, 1, 1, 2, 5, 30, 33, 64, 70, 150]) for _ in range(90)]
    lens = [n + rng.choice([0, 0, 1, 100, 128, 500, 1200]) for n in new]
    c = Case(7, 128, 2, 4, 16, e4m3, new, lens, q_scale=2.0, spare=5)
    status = i32([0])
    o, lse = (torch.full(s, 3.0, dtype=t, device="cuda") for s, t in ((c.q.shape, torch.bfloat16), (c.q.shape[:2], torch.float32)))
    c.call(o=o, lse=lse, status=status)
    assert int(status.item()) == 0
    c.check(o, lse, rows=[0, 3, 31, 32, 63, -1], heads=[0, 7])
    assert (o[c.cu[-1]:] == 3.0).all() and (lse[c.cu[-1]:] == 3.0).all()
    o2, lse2 = c.call()
    assert torch.equal(o2[:c.cu[-1]], o[:c.cu[-1]]) and torch.equal(lse2[:c.cu[-1]], lse[:c.cu[-1]])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("batch", [31, 33, 400, 1100])
def test_more_requests_than_threads(e4m3, batch):
    rng = random.Random(batch)
    new = [rng.choice([0, 1, 2, 3]) for _ in range(batch)]
    lens = [n + rng.randint(0, 60) if rng.random() < 0.9 else n for n in new]
    c = Case(batch, 64, 1, 3, 32, e4m3, new, lens, q_scale=2.0)
    o, lse = c.call()
    c.check(o, lse, requests=[b for b in range(batch) if b % max(1, batch // 40) == 0])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,new,lens", [(128, [5, 90, 200], [2, 40, 0]), (64, [200, 3, 70], [150, 0, 1]), (128, [1, 1, 64, 1], [0, 7, 0, 300])])
def test_rows_that_see_nothing(e4m3, d, new, lens):
    """Fewer tokens than new ones: the first of them see nothing and get zeros."""
    c = Case(d + sum(new), d, 1, 4, 16, e4m3, new, lens)
    status = i32([0])
    o, lse = c.call(status=status)
    assert int(status.item()) == 0
    c.check(o, lse, rows=[0, 1, 2, 3, 4, 49, 50, 51, 100, 199, -1])


def test_wild_v_scales():
    """Pages of V whose scales differ by 2^70: they are in the exponents of the weights, next to the scores."""
    c = Case(11, 128, 2, 4, 16, True, [40, 3], [400, 300], q_scale=8.0, wild=True)
    c.check(*c.call(), rows=[0, 1, 2, 20, 39])


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 1e30])
def test_extreme_queries(q_scale):
    """Rows of q of any size, of zeros and with one large value among small ones, next to e4m3 keys."""
    c = Case(13, 64, 1, 4, 32, True, [12], [100], q_scale=q_scale, k_scale=1.0 if q_scale < 1 else 1e-30)
    c.q[3] = 0.0
    c.q[4, 1, 5:] *= 1e-4
    o, lse = c.call()
    if q_scale < 1:
        c.check(o, lse)
    else:                      # scores of 1e30: a row attends to its largest one
        assert o.isfinite().all()
    for bad in (math.nan, math.inf):
        c.q[5, 2, 7] = bad
        o, lse = c.call()
        assert o[5, 2].isnan().all() and o[5, 1].isfinite().all() and o[6].isfinite().all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_out_of_range_pages_add_nothing(e4m3):
    c = Case(17, 128, 2, 3, 32, e4m3, [9, 50], [200, 400])
    c.table[0, 2], c.table[1, 0], c.table[1, 11] = -5, c.n_pages, 2 ** 31 - 1
    status = i32([0])
    o, lse = c.call(status=status)
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
    c.check(o, lse, rows=[0, 8, 30, -1], hide={(0, 2), (1, 0), (1, 11)})


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bounds", [{}, dict(max_new=6), dict(max_new=6, max_len=300000)])
def test_bad_offsets_and_lengths(e4m3, bounds):
    """A request that is not served leaves its rows alone, all others are served."""
    for batch in (5, 40):
        new, lens = [6] * batch, [60] * batch
        c = Case(batch, 64, 1, 2, 16, e4m3, new, lens)
        want = c.call(**bounds)
        for spoil in ({2: 13}, {2: -1}, {3: 1000}, {2: 9, 3: 7}):
            cu = list(c.cu)
            for i, x in spoil.items():
                cu[i] = x
            total, end, rows = c.cu[-1], 0, {}
            for b in range(batch):
                if 0 <= cu[b] <= cu[b + 1] <= total:
                    if cu[b] >= end:
                        rows[b] = (cu[b], cu[b + 1])
                    end = max(end, cu[b + 1])
            if bounds:             # one with more new tokens than announced is left out
                rows = {b: x for b, x in rows.items() if x[1] - x[0] <= 8}
            o = torch.full(c.q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
            status = i32([0])
            kvo.paged_chunk_attn(c.q, c.kp, c.vp, c.table, i32(lens), i32(cu), k_scale=c.scales[0], v_scale=c.scales[1], o=o, status=status, **bounds)
            assert int(status.item()) & kvo.DEV_BAD_COUNT or len(rows) == batch
            served = torch.zeros(total, dtype=torch.bool)
            for b, (a, e) in rows.items():
                served[a:e] = True
                if (a, e) == (c.cu[b], c.cu[b + 1]):
                    assert torch.equal(o[a:e], want[0][a:e])
            assert (o[~served.cuda()] == 3.0).all() and (o[served.cuda()] != 3.0).any()
        status = i32([0])
        o, _ = kvo.paged_chunk_attn(c.q, c.kp, c.vp, c.table, i32([-4] + [60] * (batch - 2) + [10 ** 6]), i32(c.cu), k_scale=c.scales[0],
                                    v_scale=c.scales[1], status=status, **bounds)
        assert int(status.item()) & kvo.DEV_BAD_COUNT
        assert (o[:6] == 0).all() and torch.equal(o[6:-6], want[0][6:-6])


@pytest.mark.parametrize("e4m3", [False, True])
def test_views_and_neighbours(e4m3):
    """q as a view of a fused projection, with NaN around it and in another request's rows and pages."""
    c = Case(23, 128, 2, 4, 16, e4m3, [70, 30, 200], [170, 30, 520], spare=40)
    want = c.call()
    qkv = torch.full((c.q.shape[0], 12, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    qkv[:, :8] = c.q
    qkv[c.cu[1]:c.cu[2]] = math.nan
    qkv[c.cu[-1]:] = math.nan
    for p in c.table[1, :2].tolist():
        c.kp.view(torch.uint8)[p], c.vp.view(torch.uint8)[p] = 255, 255
    o, lse = c.call(q=qkv[:, :8])
    for b in (0, 2):
        sl = slice(c.cu[b], c.cu[b + 1])
        assert torch.equal(o[sl], want[0][sl]) and torch.equal(lse[sl], want[1][sl])
    assert o[c.cu[1]:c.cu[2]].isnan().all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_token_each_is_decode_attention(e4m3):
    c = Case(29, 128, 4, 4, 32, e4m3, [1] * 6, [1, 33, 500, 128, 2000, 64])
    o, lse = c.call()
    o1, lse1 = kvo.paged_attn(c.q, c.kp, c.vp, c.table, i32(c.lens), k_scale=c.scales[0], v_scale=c.scales[1])
    c.check(o, lse, heads=[0, 15])
    c.check(o1, lse1, heads=[0, 15])


def test_a_prompt_through_the_cache_is_prompt_attention():
    """Appended in pieces and attended to piece by piece, against the whole prompt at once (bf16 both)."""
    g = torch.Generator().manual_seed(31)
    hq, hkv, d, page, n = 8, 2, 128, 32, 700
    q, k, v = ((torch.randn(n, h, d, generator=g)).bfloat16().cuda() for h in (hq, hkv, hkv))
    kp, vp = (torch.full((30, hkv, page, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.randperm(30, generator=g).int().view(1, 30).cuda()
    want, wl = kvo.prompt_attn(q, k, v, i32([0, n]))
    at = 0
    for m in (1, 128, 300, 5, 266):
        kvo.paged_append(k[at:at + m], v[at:at + m], kp, vp, table, i32([at]), cu=i32([0, m]))
        o, lse = kvo.paged_chunk_attn(q[at:at + m], kp, vp, table, i32([at + m]), i32([0, m]))
        # both round their weights once to bf16, in other units, and o once: 2 x 2^-8 of a mean of |v|, twice.  Scores of
        # sum |q k| / sqrt(d) < 16 in fp32: (d + 2) 2^-24 of that on either side
        assert (o.float() - want[at:at + m].float()).abs().max() <= 4 * ref.BF16 * v.float().abs().max()
        assert (lse - wl[at:at + m]).abs().max() <= 2 * 16 * 130 * ref.F32 + 1e-5
        at += m


def test_no_tokens():
    c = Case(1, 128, 1, 4, 16, False, [0, 0], [5, 0])
    o, lse = c.call()
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)
    empty = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 2.0)
    kvo.paged_chunk_attn(q, c.kp, c.vp, empty, i32([]), i32([0]), o=o)
    assert (o == 2.0).all()


@pytest.mark.parametrize("cap", [200, 100000])
def test_few_new_tokens_in_a_graph(cap):
    """Captured once and replayed on other offsets and lengths, whatever the workspace held before."""
    c = Case(53, 128, 2, 4, 16, True, [4, 1, 2, 4], [150, 9, 40, 200])
    lens, cu, q = i32(c.lens), i32(c.cu), c.q.clone()
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    call = lambda: kvo.paged_chunk_attn(q, c.kp, c.vp, c.table, lens, cu, k_scale=c.scales[0], v_scale=c.scales[1], max_new=4, max_len=cap, o=o,
                                        lse=lse, workspace=ws)
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for new, have in (([4, 1, 2, 4], [150, 9, 40, 200]), ([1, 1, 4, 0], [100, 5, 30, 2]), ([0, 0, 0, 4], [0, 0, 0, 131])):
        c.new, c.lens, c.cu = new, have, cuts(new)
        cu.copy_(i32(c.cu))
        lens.copy_(i32(have))
        ws.fill_(127)
        graph.replay()
        torch.cuda.synchronize()
        c.check(o, lse, heads=[0, 3, 7])


@pytest.mark.parametrize("e4m3", [False, True])
def test_streams_and_graphs(e4m3):
    """Captured into a graph and replayed on other lengths, workspaces that hold anything before, and two streams at once."""
    c = Case(37, 128, 4, 4, 64, e4m3, [30, 1, 100], [900, 3000, 100])
    other = Case(38, 128, 4, 4, 64, e4m3, [1, 40, 90], [5, 2000, 95])
    want, want_other = c.call(), other.call()
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    lens, cu, q = i32(c.lens), i32(c.cu), c.q.clone()
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    call = lambda: kvo.paged_chunk_attn(q, c.kp, c.vp, c.table, lens, cu, k_scale=c.scales[0], v_scale=c.scales[1], o=o, lse=lse, workspace=ws)
    call()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for new, have in (([30, 1, 100], [900, 3000, 100]), ([1, 1, 1], [700, 2999, 99]), ([0, 131, 0], [0, 3000, 0])):
        cu.copy_(i32(cuts(new)))
        lens.copy_(i32(have))
        ws.fill_(127)
        graph.replay()
        again = kvo.paged_chunk_attn(q, c.kp, c.vp, c.table, i32(have), i32(cuts(new)), k_scale=c.scales[0], v_scale=c.scales[1])
        n = sum(new)
        assert torch.equal(o[:n], again[0][:n]) and torch.equal(lse[:n], again[1][:n])
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append(c.call(stream=side))
        outs.append(other.call())
    torch.cuda.synchronize()
    for i, x in enumerate(outs):
        w = want_other if i % 2 else want
        assert torch.equal(x[0], w[0]) and torch.equal(x[1], w[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_pools_past_four_gigabytes(e4m3):
    hkv, page, d, n_pages = 8, 128, 128, 36000 if e4m3 else 18000        # 4.7 GB each
    dtype = E4M3 if e4m3 else torch.bfloat16
    kp, vp = (torch.zeros(n_pages, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    pages = [n_pages - 1, 1, n_pages - 2, n_pages // 2]
    g = torch.Generator().manual_seed(5)
    k, v = ((torch.randn(512, hkv, d, generator=g)).to(dtype) for _ in range(2))
    for i, p in enumerate(pages):
        kp[p], vp[p] = (x[i * page:(i + 1) * page].transpose(0, 1).cuda() for x in (k, v))
    q = torch.randn(3, 16, d, generator=g).bfloat16().cuda()
    s = torch.ones(n_pages, hkv, device="cuda") if e4m3 else None
    o, lse = kvo.paged_chunk_attn(q, kp, vp, i32([pages]), i32([500]), i32([0, 3]), k_scale=s, v_scale=s)
    for h in (0, 15):
        want, wl, tol, tl = ref.attention(q[2, h].double().cpu(), k[:500, h // 2].double(), v[:500, h // 2].double(), ref.BF16)
        extra = float(2.0 ** -17 * q[2, h].abs().max() * k[:500, h // 2].double().abs().sum(1).max() / math.sqrt(d)) if e4m3 else 0.0
        ref.check(o[2, h], want, tol + 4 * extra, f"head {h}")
