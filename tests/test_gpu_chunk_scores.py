"""Attention of new tokens over a paged cache where q, the keys or the scores are very large or very small."""
import math

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests.test_gpu_chunk import Case, i32
from tests.test_gpu_chunk_scales import check, rescale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("q_scale,k_log", [(1e30, -107), (1e36, -126), (2e-30, 90), (1e-36, 110), (1e-3, 3)])
def test_ordinary_scores_of_extreme_factors(q_scale, k_log, few):
    """Rows of q of any size next to e4m3 keys whose scale is as small or as large: scores of some units."""
    c = Case(13, 64, 1, 4, 32, True, [4 if few else 12], [100], q_scale=q_scale)
    rescale(c, k=lambda b, i: 2.0 ** k_log)
    c.q[3] = 0.0
    c.q[2, 1, 5:] *= 1e-4
    o, lse = c.call(max_new=4 if few else 0)
    check(c, o, lse, range(12), range(4))
    spread = (c.rows[0][0][:, 0] @ c.q[0, 0].double().cpu() / 8).std()
    assert 0.1 < float(spread) < 1000          # (the scores do matter)


class Steep:
    """Keys whose scores are whole multiples of a unit of 2^a (q has one value, keys whole numbers there): each row's softmax is the
    mean over the keys with its largest score."""

    def __init__(self, a, sign, e4m3, new, lens, seed, one_scale):
        self.c = c = Case(seed, 64, 1, 4, 16, e4m3, new, lens)
        g = torch.Generator().manual_seed(seed)
        # few keys have the largest number, and the rows before them do not see them
        self.codes = [sign * torch.randint(1, 9, (n,), generator=g).float() + (0 if sign > 0 else -1) for n in lens]
        self.a = a
        for b, n in enumerate(lens):
            for t in range(n):
                c.kp[int(c.table[b, t // 16]), 0, t % 16, 0] = float(self.codes[b][t])
        if e4m3:
            rescale(c, k=lambda b, i: 1.0, v=(lambda b, i: 0.25) if one_scale else (lambda b, i: 2.0 ** (i % 4 - 3)))
        c.q.zero_()
        c.q[..., 0] = 2.0 ** (a + 3)           # over sqrt(64)

    def check(self, o, lse, exact):
        c = self.c
        for b, (n, have) in enumerate(zip(c.new, c.lens)):
            for i in range(n):
                see = have - n + i + 1
                k = self.codes[b][:see]
                top = k == k.max()
                v = c.rows[1][b][:see, 0][top]
                got = o[c.cu[b] + i].double().cpu()
                room = 2.0 ** -8 * v.abs().max(0).values + 2.0 ** -8 * v.mean(0).abs() + 1e-30        # weights to bf16, o to bf16
                assert (got <= v.max(0).values + room).all() and (got >= v.min(0).values - room).all(), (b, i)
                if exact:
                    assert ((got - v.mean(0)).abs() <= room).all(), (b, i)
                want = float(k.max()) * 2.0 ** self.a
                # the score, its factor of log2(e) and back, and the count, in fp32
                assert ((lse[c.cu[b] + i].double().cpu() - want - math.log(int(top.sum()))).abs() <= abs(want) * 2.0 ** -21 + 2.0 ** -18).all()


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("a", [8, 14, 17, 20, 21, 22, 23, 24, 25, 26, 27, 28, 30, 40, 60, 100, 120])
def test_scores_of_any_size(a, sign, e4m3, few):
    """2^20 and beyond: fp32's steps there are no longer small next to 1."""
    new, lens = ([4, 2], [300, 40]) if few else ([40, 6], [300, 40])
    for one_scale in (True, False) if e4m3 else (True,):
        s = Steep(a, sign, e4m3, new, lens, a + 2 * e4m3, one_scale)
        status = i32([0])
        o, lse = s.c.call(max_new=4 if few else 0, status=status)
        assert int(status.item()) == 0
        s.check(o, lse, exact=one_scale)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("a", [0, 12, 19, 22, 24, 25, 26, 27, 28, 29, 30, 34])
def test_large_scores_that_lie_close(a, e4m3, few):
    """Scores of 2^a plus small ones: fp32 holds them to 2^(a - 24), and o is a mean of the values whatever is left of them."""
    for seed in range(6):
        c = Case(100 * a + seed, 64, 1, 4, 16, e4m3, [4 if few else 30], [500], q_scale=1.0)
        c.kp[..., 0] = 1.0
        c.rows[0][0][..., 0] = 1.0
        if e4m3:
            rescale(c, k=lambda b, i: 2.0 ** -5, v=lambda b, i: 2.0 ** -7)
        c.q[..., 0] = 2.0 ** (a + (8 if e4m3 else 3))
        o, lse = c.call(max_new=4 if few else 0)
        v = c.rows[1][0][:, 0]
        assert o.isfinite().all() and (o.double().cpu().abs() <= v.abs().max(0).values * (1 + 2.0 ** -7)).all()
        # log2(e) times the score is rounded to fp32, and the logarithm of 500 keys' weights and their scores of up to 100 are added
        assert ((lse - 2.0 ** a).abs() <= 2.0 ** (a - 21) + 120).all()
        if a < 4:
            check(c, o, lse, [0, 1, -1], [0, 3])


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("less", [21, 22, 23, 24])
@pytest.mark.parametrize("a", list(range(19, 32)))
def test_scores_one_step_apart(a, less, e4m3, few):
    """Scores of 2^a, and later ones that are larger by 0 to 7 times 2^(a - less): some steps of fp32, so that a rise of the running
    maximum by just what is let pass comes up; the weights are still those of fp32's scores, so o is a mean of the values."""
    for sign in (1, -1):
        c = Case(a, 64, 1, 4, 16, e4m3, [4 if few else 30], [600], q_scale=1.0)
        c.q.zero_()
        c.kp[..., :2] = 0.0
        # (factors that q's two e4m3 values hold exactly: 2^8 and 2^-9 in the keys, 2^-4 to 2^-7 in q)
        c.kp[..., 0] = 2.0 ** 8
        for t in range(600):
            c.kp[int(c.table[0, t // 16]), 0, t % 16, 1] = float(t * 8 // 600) * 2.0 ** -9
        if e4m3:
            rescale(c, k=lambda b, i: 1.0, v=lambda b, i: 2.0 ** -7)
        c.q[..., 0] = sign * 2.0 ** (a + 3 - 8)
        c.q[..., 1] = 2.0 ** (a + 3 - 8 - (less - 17))
        o, lse = c.call(max_new=4 if few else 0)
        v = c.rows[1][0][:, 0]
        assert o.isfinite().all() and (o.double().cpu().abs() <= v.abs().max(0).values * (1 + 2.0 ** -7)).all()
        # the largest score, log2(e) times it in fp32, and the logarithm of at most 600 weights
        assert ((lse - sign * 2.0 ** a - 7 * 2.0 ** (a - less)).abs() <= 2.0 ** (a - 21) + 7).all()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("less", [22, 23, 24])
@pytest.mark.parametrize("a", list(range(22, 31)))
def test_scores_one_step_apart_for_few_rows(a, less, e4m3, decode):
    """The same with many tiles of keys to a warp of the kernels for few rows: 128 requests over the same pages."""
    n, page, b = 8000, 64, 128
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    g = torch.Generator().manual_seed(a)
    k = torch.zeros(n, 64)
    k[:, 0], k[:, 1] = 1.0, (torch.arange(n) * 64 // n).float() % 8 + (torch.arange(n) * 8 // n).float()
    v = torch.randn(n, 64, generator=g).to(dtype)
    kp, vp = (x.view(n // page, 1, page, 64).cuda() for x in (k.to(dtype), v))
    table = i32(list(range(n // page))).view(1, -1).repeat(b, 1).contiguous()
    q = torch.zeros(b, 4, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 1] = 2.0 ** (a + 3), 2.0 ** (a + 3 - less)
    one = torch.ones(n // page, 1, device="cuda") if e4m3 else None
    lens = i32([n] * b)
    if decode:
        o, lse = kvo.paged_attn(q, kp, vp, table, lens, k_scale=one, v_scale=one)
    else:
        o, lse = kvo.paged_chunk_attn(q, kp, vp, table, lens, i32(list(range(b + 1))), k_scale=one, v_scale=one, max_new=1)
    assert o.isfinite().all() and (o.double().cpu().abs() <= v.double().abs().max() * (1 + 2.0 ** -7)).all()
    assert ((lse - 2.0 ** a - 14 * 2.0 ** (a - less)).abs() <= 2.0 ** (a - 21) + 9).all()


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [math.inf, math.nan, "overflow"])
def test_scores_that_are_not_finite(bad, e4m3, few):
    """Rows that see such a score are NaN, o and lse; rows before that key are as they were."""
    if e4m3 and bad == math.inf:
        pytest.skip("e4m3 has no infinity")
    new, lens = ([4, 2], [300, 40]) if few else ([40, 6], [300, 40])
    kw = dict(max_new=4 if few else 0)
    for at in (lens[0] - 2, 0, 130):               # the last token but one, the first, and one in the middle
        c = Case(5, 64, 1, 4, 16, e4m3, new, lens)
        c.q[..., 3] = c.q[..., 3].abs() + 1.0
        want = c.call(**kw)
        page, row = int(c.table[0, at // 16]), at % 16
        if bad == "overflow":                      # 2^30 times the other scores, and those near fp32's largest number
            if e4m3:                               # (a scale is its whole page's: the other keys there become 0)
                c.kp[page] = 0.0
                c.scales[0][page] = 2.0 ** 26
            c.kp[page, 0, row, 3] = 448.0 if e4m3 else 3e38
            c.q[..., 3] *= 2.0 ** 100
            want = None
        else:
            c.kp.view(torch.uint8 if e4m3 else torch.bfloat16)[page, 0, row, 3] = 0x7F if e4m3 else bad
        o, lse = c.call(**kw)
        first = max(at - (lens[0] - new[0]), 0)
        if want is not None:
            assert torch.equal(o[:first], want[0][:first]) and torch.equal(lse[:first], want[1][:first])
            assert torch.equal(o[new[0]:], want[0][new[0]:]) and torch.equal(lse[new[0]:], want[1][new[0]:])
        else:
            assert o[:first].isfinite().all() and o[new[0]:].isfinite().all()
        assert o[first:new[0]].isnan().all() and not lse[first:new[0]].isfinite().any()


@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_score_in_a_row_of_its_own(d):
    """The first score that a row's maximum takes up, and the last: many requests, most in one range of the plan."""
    n = 700
    kp, vp = (torch.randn(40, 1, 16, d, generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in (1, 2))
    kp[2, 0, 6, 3] = math.inf                      # token 38 of every request
    q = torch.randn(n * 40, 4, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q[..., 3] = q[..., 3].abs() + 0.5
    o, lse = kvo.paged_chunk_attn(q, kp, vp, i32([[0, 1, 2]] * n), i32([40] * n), i32([40 * b for b in range(n + 1)]))
    o, lse = o.view(n, 40, 4, d), lse.view(n, 40, 4)
    assert o[:, 38:].isnan().all() and not lse[:, 38:].isfinite().any()
    assert o[:, :38].isfinite().all() and lse[:, :38].isfinite().all()
