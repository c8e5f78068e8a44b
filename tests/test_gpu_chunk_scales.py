"""Attention of new tokens over e4m3 pages whose scales are very small, very large or far apart, against 64 bits."""
import math
import random

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests import paged_ref as ref
from tests.test_gpu_chunk import Case, i32

pytestmark = pytest.mark.gpu


def rescale(c, v=None, k=None):
    """Page i of request b gets the scales v(b, i) and k(b, i) in all heads; `None`: as they are."""
    need = [-(-n // c.page) for n in c.lens]
    for which, (scale, pool, f) in enumerate(zip(c.scales, (c.kp, c.vp), (k, v))):
        if f is None:
            continue
        for b, n in enumerate(need):
            for i in range(n):
                scale[int(c.table[b, i])] = f(b, i)
        for b, n in enumerate(need):
            ids = c.table[b, :n].long()
            x = pool[ids].double() * scale[ids].double()[..., None, None]
            c.rows[which][b] = x.transpose(1, 2).reshape(n * c.page, c.hkv, c.d)[:c.lens[b]].cpu()


def check(c, o, lse, rows, heads, unit=1.0):
    """Rows against 64 bits, in units of `unit` (an absolute bound means nothing next to values of 2^-120)."""
    for b, (n, have) in enumerate(zip(c.new, c.lens)):
        need = -(-have // c.page)
        for i in sorted({x % n for x in rows if n}):
            see = max(have - n + i + 1, 0)
            for h in heads:
                g = h // c.r
                q = c.q[c.cu[b] + i, h].double().cpu()
                k, v = c.rows[0][b][:see, g], c.rows[1][b][:see, g] / unit
                want, wl, tol, tl = ref.attention(q, k, v, 2 * ref.BF16)
                s = k @ q / math.sqrt(c.d)
                w = torch.softmax(s, 0)
                scale = c.scales[1][c.table[b, :need].long(), g].double().cpu() if c.e4m3 else torch.ones(need, dtype=torch.float64)
                scale = scale.repeat_interleave(c.page)[:see]
                log = torch.log2(scale.clamp(min=2.0 ** -160))
                # q as two e4m3 values, each within 2^-17 of the row's largest; the scores' logarithms with v_scale's in them,
                # in fp32: the product, the maximum, their difference and the sum's unit, half a step of the largest each
                ds = float(2.0 ** -17 * q.abs().max() * k.abs().sum(1).max() / math.sqrt(c.d))
                size = float((s.abs().max() / math.log(2) + log.abs().max()) * 2 + 8)
                ds += 4 * ref.F32 * size * math.log(2)
                tol = tol + 2 * ds * (w @ v.abs())
                # weights times v_scale have steps of 2^-30 of the largest of them: half a step to a key, times a code
                tol = tol + see * 2.0 ** -31 * float((w * scale).max()) / unit * 448
                tol = tol + 2.0 ** -134 / unit + 2.0 ** -148 / unit        # the steps of values below bf16's (fp32's) normal ones
                ref.check(o[c.cu[b] + i, h].double() / unit, want, tol, f"o of request {b}, token {i}, head {h}")
                got = float(lse[c.cu[b] + i, h])
                assert abs(got - wl) <= tl + ds, (b, i, h, got, wl)


@pytest.mark.parametrize("log", [-126, -123, -120, -118, -115, -107, -100, -64, 64, 100, 117])
@pytest.mark.parametrize("d,new,lens", [(128, [20, 40], [300, 2100]), (64, [30], [20000]), (128, [200, 9, 1], [200, 140, 128])])
def test_one_scale(log, d, new, lens):
    """All pages alike: 20 to 40 tokens are one tile of rows or two, 20000 keys are cut by the CTAs' ranges."""
    c = Case(d + len(lens), d, 1, 4, 32, True, new, lens, q_scale=0.5)
    rescale(c, v=lambda b, i: 2.0 ** log)
    status = i32([0])
    o, lse = c.call(status=status)
    assert int(status.item()) == 0
    check(c, o, lse, [0, 1, 17, -1], [0, 3], unit=2.0 ** log)


@pytest.mark.parametrize("cap", [0, 100000])
@pytest.mark.parametrize("log", [-100, -64, 64, 80])
def test_one_scale_and_few_rows(log, cap):
    """The kernels of up to 16 rows, in their range of scales: 2^-100 to 2^100 over the tokens."""
    c = Case(7, 128, 1, 4, 32, True, [4, 1], [300, 2100], q_scale=0.5)
    rescale(c, v=lambda b, i: 2.0 ** log)
    o, lse = c.call(max_new=4, max_len=max(cap, 2100))
    check(c, o, lse, [0, 1, 2, 3], [0, 3], unit=2.0 ** log)


def test_scales_of_zero():
    """Pages of V that are zero whatever their codes: next to others, they take part in the softmax; alone, o is zero."""
    c = Case(3, 128, 1, 4, 16, True, [20, 40], [300, 700])
    rescale(c, v=lambda b, i: 0.0 if (b + i) % 2 else 0.5)
    o, lse = c.call()
    check(c, o, lse, [0, 7, -1], [0, 3])
    rescale(c, v=lambda b, i: 0.0)
    o, lse = c.call()
    assert (o == 0).all()
    check(c, o, lse, [0, 7, -1], [0, 3])


def test_pages_of_zeros_that_lead():
    """What an append of zeros leaves, codes of 0 next to a scale of 2^-100, where such pages hold most of the softmax."""
    c = Case(5, 128, 1, 4, 16, True, [20, 40], [300, 700])
    lead = lambda b, i: i % 3 == 1
    for b in range(2):
        for i in range(-(-c.lens[b] // c.page)):
            if lead(b, i):
                m = min(c.page, c.lens[b] - i * c.page)
                c.vp.view(torch.uint8)[int(c.table[b, i]), :, :m] = 0
    for power in (0, 2, 4, 6, 8):
        rescale(c, v=lambda b, i: 2.0 ** -100 if lead(b, i) else 0.25, k=lambda b, i: 2.0 ** (power - 8) if lead(b, i) else 2.0 ** -8)
        o, lse = c.call()
        check(c, o, lse, [0, 7, 15, -1], [0, 3])


LOGS = [[-126, 0, 100], [-100, -3], [110, -126], [-40, 40], [0, 33, -33], [-126, -126, -126, 117], [20, 52, 84, 116], [0, -32, -64, -96, -126],
        [-3] * 9 + [90] + [-3] * 9 + [-120]]


@pytest.mark.parametrize("order", ["as it is", "reversed", "shuffled"])
@pytest.mark.parametrize("logs", LOGS)
@pytest.mark.parametrize("d,new,lens", [(128, [20], [300]), (64, [50, 3], [700, 390]), (128, [10], [9000])])
def test_scales_far_apart(logs, order, d, new, lens):
    """Scores that differ by up to hundreds next to scales that differ by up to 2^243: either may lead."""
    rng = random.Random(f"{logs} {order} {d}")
    for steep in (0, 3, 7):
        c = Case(d + steep, d, 1, 4, 16, True, new, lens, q_scale=1.0)
        runs = rng.choice([1, 5, 8, 24])               # pages in a row of one scale
        need = -(-max(lens) // c.page)
        log = [logs[i // runs % len(logs)] for i in range(need)]
        if order == "reversed":
            log.reverse()
        elif order == "shuffled":
            rng.shuffle(log)
        kick = [rng.choice([0, steep]) for _ in range(need)]
        rescale(c, v=lambda b, i: 2.0 ** log[i], k=lambda b, i: 2.0 ** (kick[i] - 9) * 1.25)
        status = i32([0])
        o, lse = c.call(status=status)
        assert int(status.item()) == 0
        check(c, o, lse, [0, 3, -1], [0, 3], unit=2.0 ** min(logs))
        again = c.call()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
