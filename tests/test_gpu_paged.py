"""Rotary positions, the paged cache (bf16 and e4m3) and the attention over it, against plain 64-bit references."""
import math

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("tokens,heads,d,rot,interleaved,scaling", [
    (1, 1, 64, 64, False, None), (1, 40, 128, 128, True, "banded"), (5, 3, 128, 64, False, "linear"),
    (37, 10, 128, 128, False, "ramp"), (33, 5, 64, 16, True, None), (6, 2, 48, 32, False, None),
    (4, 1, 256, 256, True, "banded"), (300, 48, 128, 96, False, None)])
def test_rope_matches_reference(tokens, heads, d, rot, interleaved, scaling):
    g = gen(tokens * 1000 + heads)
    freq, amp = kvo.rope_frequencies(rot, 500000.0, scaling, factor=8.0)
    x = normal(g, tokens, heads, d)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1 if tokens > 1 else 131071
    if tokens > 2:
        pos[1], pos[2] = 0, -77777
    y = kvo.rope(x, pos.cuda(), freq, interleaved, amp)
    n = min(tokens, 40)
    want, mag = ref.rope(x[:n], pos[:n], freq, interleaved, amp)
    ref.check(y[:n], want, ref.rope_bound(want, mag), "rope")
    assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_strides_and_in_place():
    """q and k heads of a fused projection, a head-major buffer, in place, and a single token of odd strides."""
    g = gen(5)
    freq, amp = kvo.rope_frequencies(128)
    pos = i32([3, 70000, 12, 9, 9])
    qkv = normal(g, 5, 12, 128)
    want = kvo.rope(qkv[:, 2:9].contiguous(), pos, freq)
    assert torch.equal(kvo.rope(qkv[:, 2:9], pos, freq), want)
    head_major = qkv[:, 2:9].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(kvo.rope(head_major, pos, freq), want)
    before = qkv.clone()
    assert kvo.rope(qkv[:, 2:9], pos, freq, out=qkv[:, 2:9]).data_ptr() == qkv[:, 2:9].data_ptr()
    assert torch.equal(qkv[:, 2:9], want)
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 9:], before[:, 9:])
    assert kvo.rope(qkv[:0], pos[:0], freq).shape == (0, 12, 128)
    # turning by p, then by -p, comes back to within the two roundings
    x = before[:, 2:9].float()
    back = kvo.rope(want, -pos, freq).float()
    pair = x.abs() + x.roll(64, -1).abs()
    assert ((back - x).abs() <= 2 * 2.0 ** -8 * pair + 2.0 ** -19 * pair).all()


# ------------------------------------------------------------------ append
def pools(g, n_pages, hkv, page, d, e4m3):
    """Pools full of stale bytes (NaN codes among them), scales full of NaN."""
    if not e4m3:
        k, v = normal(g, n_pages, hkv, page, d), normal(g, n_pages, hkv, page, d)
        k[0] = math.nan
        return k, v, None, None
    raw = [torch.randint(0, 256, (n_pages, hkv, page, d), generator=g, dtype=torch.uint8).cuda().view(E4M3)
           for _ in range(2)]
    scale = [torch.full((n_pages, hkv), math.nan, device="cuda") for _ in range(2)]
    return raw[0], raw[1], scale[0], scale[1]


def bytes_of(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().clone()


def pow2_scale(amax):
    s = 2.0 ** -100
    while s * 448.0 < amax:
        s *= 2
    return s


def expect_append(raw, scale, x, table, start, cu, page):
    """The pool's bytes (and scales) after appending the bf16 rows x, by the definition."""
    for b in range(len(start)):
        at, end = start[b], start[b] + cu[b + 1] - cu[b]
        while at < end:
            p, lo, n = table[b][at // page], at % page, min(page - at % page, end - at)
            rows = x[cu[b] + at - start[b]:cu[b] + at - start[b] + n]
            for h in range(x.shape[1]):
                if scale is None:
                    raw[p, h, lo:lo + n] = rows[:, h].view(torch.int16)
                    continue
                r = rows[:, h].float()
                fin = r[torch.isfinite(r)]
                s = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                if lo:
                    old = float(scale[p, h])
                    s = max(s, old)
                    raw[p, h, :lo] = (raw[p, h, :lo].view(E4M3).float() * (old / s)).to(E4M3).view(torch.uint8)
                scale[p, h] = s
                r = torch.where(torch.isfinite(r), r, torch.full_like(r, math.nan))
                raw[p, h, lo:lo + n] = (r * (1.0 / s)).to(E4M3).view(torch.uint8)
            at += n


def same_bytes(got, want, what):
    """Equal bytes, any NaN code of e4m3 equal to any other."""
    nan = lambda t: (t & 0x7F) == 0x7F if t.dtype == torch.uint8 else torch.zeros_like(t, dtype=torch.bool)
    bad = (got != want) & ~(nan(got) & nan(want))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,hkv,hq,page,counts,starts,rot,interleaved", [
    (128, 2, 8, 16, [1, 1, 1], [0, 15, 16], 128, False),          # decode: a page begun, filled, begun again
    (64, 1, 1, 32, [1], [31], 32, True),
    (128, 1, 3, 64, [70, 0, 1, 200], [3, 5, 63, 0], 64, False),    # ragged prompts, one request without tokens
    (64, 3, 6, 128, [129, 257], [127, 1], 64, True),
    (128, 2, 2, 128, [300], [0], 0, False),                       # no rotation
    (64, 8, 16, 16, [17] * 40, list(range(40)), 48, False)])
def test_append_matches_definition(e4m3, d, hkv, hq, page, counts, starts, rot, interleaved):
    g = gen(page + d + len(counts))
    b, tokens = len(counts), sum(counts)
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    per = [(s + n + page - 1) // page for s, n in zip(starts, counts)]
    n_pages = sum(per) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    table = [[order.pop() for _ in range(p)] + [0] * (max(per) - p) for p in per]
    kp, vp, ks, vs = pools(g, n_pages, hkv, page, d, e4m3)
    if e4m3:      # pages that the requests have begun hold values of a known scale, some too small for what comes
        for i, s in enumerate(starts):
            if s % page:
                p = table[i][s // page]
                for sc, pool in ((ks, kp), (vs, vp)):
                    sc[p] = torch.tensor([2.0 ** (-20 + 9 * ((i + h) % 3)) for h in range(hkv)]).cuda()
                    pool[p].copy_((torch.randn(hkv, page, d, generator=g) * 90).clamp(-448, 448).to(E4M3).cuda())
    wide = normal(g, tokens + 3, hq + 2 * hkv, d)                  # a fused projection with padding rows behind
    q, k, v = wide[:tokens, :hq], wide[:tokens, hq:hq + hkv], wide[:tokens, hq + hkv:]
    freq = kvo.rope_frequencies(rot, 10000.0)[0] if rot else None
    k_out = torch.full((tokens, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_k, want_v = bytes_of(kp), bytes_of(vp)
    want_ks, want_vs = (ks.cpu(), vs.cpu()) if e4m3 else (None, None)
    one = all(n == 1 for n in counts)
    for again in range(2):        # the same rows again: nothing changes
        q_out = kvo.paged_append(k, v, kp, vp, i32(table), i32(starts), cu=None if one else i32(cu), k_scale=ks,
                                 v_scale=vs, freq=freq, interleaved=interleaved, q=q, k_out=k_out, status=status)
        assert int(status.item()) == 0
        if again:
            assert torch.equal(bytes_of(kp), first[0]) and torch.equal(bytes_of(vp), first[1])
            break
        first = bytes_of(kp), bytes_of(vp)
        pos = torch.cat([torch.arange(n) + s for n, s in zip(counts, starts)])
        if rot:
            want, mag = ref.rope(k, pos, freq, interleaved, 1.0)
            ref.check(k_out, want, ref.rope_bound(want, mag), "k_out")
            assert torch.equal(q_out, kvo.rope(q, pos.int().cuda(), freq, interleaved))
        else:
            assert torch.equal(k_out, k) and torch.equal(q_out, q)
        expect_append(want_k, want_ks, k_out.cpu(), table, starts, cu, page)
        expect_append(want_v, want_vs, v.cpu(), table, starts, cu, page)
        same_bytes(bytes_of(kp), want_k, "k pages")
        same_bytes(bytes_of(vp), want_v, "v pages")
        if e4m3:
            assert torch.equal(torch.nan_to_num(ks.cpu(), -1.0), torch.nan_to_num(want_ks, -1.0))
            assert torch.equal(torch.nan_to_num(vs.cpu(), -1.0), torch.nan_to_num(want_vs, -1.0))


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_append_of_many_short_requests(e4m3, d, page):
    """Several heads to a CTA, each kind of page: rows begun, a page's border passed, heads left over for the last CTA."""
    counts, starts = [(5 * i) % 9 + 1 for i in range(70)], [(29 * i) % (2 * page) for i in range(70)]
    test_append_matches_definition(e4m3, d, 7, 14, page, counts, starts, d // 2, d == 64)


def test_append_extreme_values():
    """Zeros, the largest bf16, subnormals, infinities and NaN: scales from the finite values, NaN codes for the rest."""
    rows = torch.zeros(6, 1, 64)
    rows[1, 0, 0] = 3.3e38
    rows[2, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    rows[2, 0, 3] = 448.0
    rows[3, 0, 5] = 1e-39
    rows[4, 0, 7] = 449.0 * 2 ** -9
    rows[5, 0, :2] = torch.tensor([448.0, 2.0 ** -9])
    x = rows.bfloat16().cuda()
    kp, vp, ks, vs = pools(gen(1), 6, 1, 16, 64, True)
    kvo.paged_append(x, x, kp, vp, i32([[i] for i in range(6)]), i32([0] * 6), k_scale=ks, v_scale=vs)
    want, want_s = bytes_of(kp), torch.full((6, 1), math.nan)
    expect_append(want, want_s, x.cpu(), [[i] for i in range(6)], [0] * 6, list(range(7)), 16)
    same_bytes(bytes_of(kp), want, "k pages")
    same_bytes(bytes_of(vp)[:, :, :1], bytes_of(kp)[:, :, :1], "v pages")
    assert torch.equal(ks.cpu(), want_s) and torch.equal(vs.cpu(), want_s)
    assert float(ks[0]) == 2.0 ** -100 and float(ks[2]) == 1.0


def test_append_skips_what_is_out_of_range():
    """Bad page ids, tokens past the table and bad offsets: a status bit, the rest of the call unharmed."""
    g = gen(3)
    k = normal(g, 4, 1, 64)
    for table, start, cu, bit in [([[0], [9], [1], [-1]], [0, 0, 0, 0], None, kvo.DEV_BAD_BLOCK_ID),
                                  ([[0], [2], [1], [3]], [0, 16, 0, -5], None, kvo.DEV_BAD_COUNT),
                                  ([[0], [1]], [0, 0], [0, 2, 9], kvo.DEV_BAD_COUNT),
                                  ([[0], [1]], [0, 0], [0, 3, 1], kvo.DEV_BAD_COUNT)]:
        kp, vp, ks, vs = pools(g, 4, 1, 16, 64, True)
        before = bytes_of(kp)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full((4, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        kvo.paged_append(k, k, kp, vp, i32(table), i32(start), cu=None if cu is None else i32(cu), k_scale=ks,
                         v_scale=vs, q=k, q_out=q_out, status=status)
        assert int(status.item()) == bit
        after = bytes_of(kp)
        good = [0, 1] if cu is None and bit == kvo.DEV_BAD_BLOCK_ID else [0, 1] if cu is None else [0]
        assert (after[0, 0, 0] != before[0, 0, 0]).any()
        for p in set(range(4)) - set(good):
            assert torch.equal(after[p], before[p])


# ------------------------------------------------------------------ attention
def cache_of(g, lens, hkv, page, d, e4m3, spare=1):
    """Pools whose rows behind each request's last token are NaN, scales of several binades, and the 64-bit rows."""
    need = [max(1, (n + page - 1) // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).tolist()
    table = [[order.pop() for _ in range(p)] + [order[0]] * (max(need) - p) for p in need]
    scale = [None, None]
    if e4m3:
        pool = [(torch.randn(n_pages, hkv, page, d, generator=g) * 100).clamp(-448, 448).to(E4M3) for _ in range(2)]
        scale = [torch.exp2(torch.randint(-9, -5, (n_pages, hkv), generator=g).float()) for _ in range(2)]
        scale[1][0] *= 1.37                                        # a scale that is no power of two is allowed
        full = [p.double() * s.double()[..., None, None] for p, s in zip(pool, scale)]
    else:
        pool = [torch.randn(n_pages, hkv, page, d, generator=g).bfloat16() for _ in range(2)]
        full = [p.double() for p in pool]
    rows = []
    for i, n in enumerate(lens):
        at = torch.tensor(table[i][:(n + page - 1) // page], dtype=torch.long)
        rows.append([f[at].transpose(0, 1).flatten(1, 2)[:, :n] for f in full])
        last = table[i][(n - 1) // page] if n else None
        if n and n % page:
            for p in pool:
                p.view(torch.uint8 if e4m3 else torch.int16)[last, :, n % page:] = 0x7F if e4m3 else 0x7FC0
    to = lambda t: None if t is None else t.cuda()
    return [to(p) for p in pool], [to(s) for s in scale], i32(table), rows


def check_attention(q, got, rows, hkv, weight, pick=None):
    o, lse = got
    r = q.shape[1] // hkv
    for b, (k, v) in enumerate(rows):
        for h in range(q.shape[1]):
            kk, vv = k[h // r], v[h // r]
            if pick is not None:
                kk, vv = kk[pick[b][h // r]], vv[pick[b][h // r]]
            want, wl, tol, tl = ref.attention(q[b, h].double().cpu(), kk, vv, weight)
            ref.check(o[b, h], want, tol, f"o[{b}][{h}]")
            assert float(lse[b, h]) == wl or abs(float(lse[b, h]) - wl) <= tl, (b, h, float(lse[b, h]), wl)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,hkv,r,page,lens", [
    (128, 1, 1, 16, [1]), (64, 1, 1, 16, [1]), (128, 2, 4, 32, [0, 33, 16, 100]), (64, 2, 4, 16, [4096]),
    (128, 1, 16, 64, [2500, 7]), (64, 3, 9, 128, [129, 0, 640, 1]), (128, 8, 4, 64, [700, 1, 513]),
    (64, 1, 5, 32, [15, 16, 17, 31, 32, 33, 63, 64, 65] * 3), (128, 1, 2, 16, [0, 0]), (128, 1, 8, 128, [9000])])
def test_paged_attention_matches_reference(e4m3, d, hkv, r, page, lens):
    g = gen(d + r + len(lens))
    (kp, vp), (ks, vs), table, rows = cache_of(g, lens, hkv, page, d, e4m3)
    q = normal(g, len(lens), hkv * r, d, scale=1.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # a table of a long capacity (and no bound on the lengths) is cut into ranges, a short one into clusters
    long = torch.zeros(len(lens), 120000 // page, dtype=torch.int32, device="cuda")
    long[:, :table.shape[1]] = table
    for tb, max_len in ((table, 0), (table, max(max(lens), 1)), (long, 0), (long, 300)):
        for again in range(2):
            got = kvo.paged_attn(q, kp, vp, tb, i32(lens), k_scale=ks, v_scale=vs, max_len=max_len, status=status)
            if again:
                assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
            first = got
        check_attention(q, got, rows, hkv, ref.F16 if e4m3 else ref.BF16)
    assert int(status.item()) == 0


@pytest.mark.parametrize("d,e4m3", [(128, True), (64, False), (64, True), (128, False)])
@pytest.mark.parametrize("groups,r", [(390, 8), (200, 5), (133, 8), (100, 1), (66, 8), (50, 3), (33, 8), (18, 7), (280, 9), (140, 16),
                                      (93, 11), (70, 16), (46, 16), (35, 13), (23, 16), (12, 16)])
def test_paged_attention_in_clusters_of_every_size(groups, r, d, e4m3):
    """1 to 16 CTAs a group (as many as fit for so many groups), most of whose warps have no tile."""
    g = gen(groups + r)
    lens = [(37 * i) % 71 for i in range(groups)]
    lens[groups // 2], lens[-1] = 900, 300
    (kp, vp), (ks, vs), table, rows = cache_of(g, lens, 1, 16, d, e4m3)
    bound = 1500 if groups > 200 else 2100        # more than 15 x 128 tokens may take 16 CTAs, more than 1536 need two
    wide = torch.zeros(groups, 140, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = normal(g, groups, r, d, scale=1.5)
    got = kvo.paged_attn(q, kp, vp, wide, i32(lens), k_scale=ks, v_scale=vs, max_len=bound)
    keep = sorted({0, 1, 2, 5, groups // 3, groups // 2, groups - 2, groups - 1})
    check_attention(q[keep], (got[0][keep], got[1][keep]), [rows[i] for i in keep], 1, ref.F16 if e4m3 else ref.BF16)
    again = kvo.paged_attn(q, kp, vp, wide, i32(lens), k_scale=ks, v_scale=vs, max_len=bound)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    # as ranges
    long = torch.zeros(groups, 120000 // 16, dtype=torch.int32, device="cuda")
    long[:, :table.shape[1]] = table
    other = kvo.paged_attn(q, kp, vp, long, i32(lens), k_scale=ks, v_scale=vs)
    check_attention(q[keep], (other[0][keep], other[1][keep]), [rows[i] for i in keep], 1, ref.F16 if e4m3 else ref.BF16)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,hkv,r,page,n_blocks,lens", [
    (128, 2, 4, 32, 3, [300, 70]), (64, 1, 8, 16, 40, [700, 3, 0]), (128, 4, 1, 64, 12, [1500]), (64, 1, 3, 64, 600, [900, 64])])
def test_paged_attention_over_listed_blocks(e4m3, d, hkv, r, page, n_blocks, lens):
    """Each KV head its own blocks, a cut last one, one past the end, one twice, and counts of every size."""
    g = gen(n_blocks)
    (kp, vp), (ks, vs), table, rows = cache_of(g, lens, hkv, page, d, e4m3)
    have = table.shape[1]
    blocks = torch.randint(0, have, (len(lens), hkv, n_blocks), generator=g, dtype=torch.int32)
    blocks[0, 0, 0] = (lens[0] - 1) // page
    blocks[0, 0, -1] = blocks[0, 0, 0]
    counts = torch.randint(0, min(n_blocks, 40) + 1, (len(lens), hkv), generator=g, dtype=torch.int32)
    counts[0, 0] = min(n_blocks, 40)
    counts[-1, -1] = 0
    for cnt in (None, counts):
        pick = []
        for b, n in enumerate(lens):
            pick.append([])
            for h in range(hkv):
                use = blocks[b, h, :n_blocks if cnt is None else int(cnt[b, h])].tolist()
                pick[-1].append(torch.tensor([t for x in use for t in range(x * page, min(n, (x + 1) * page))],
                                             dtype=torch.long))
        q = normal(g, len(lens), hkv * r, d)
        got = kvo.paged_attn(q, kp, vp, table, i32(lens), k_scale=ks, v_scale=vs, blocks=blocks.cuda(),
                             counts=None if cnt is None else cnt.cuda())
        check_attention(q, got, rows, hkv, ref.F16 if e4m3 else ref.BF16, pick)


def test_paged_attention_extreme_scores():
    """Scores far apart (the maximum rises late), a q row of zeros, large and tiny q, NaN in an attended key."""
    g = gen(11)
    lens, d, page = [400, 400, 400, 400, 64], 64, 16
    (kp, vp), (ks, vs), table, rows = cache_of(g, lens, 1, page, d, True)
    q = normal(g, 5, 2, d)
    q[0] *= 60.0
    q[1] = 0.0
    q[2] *= 1e-20
    q[3, 0], q[3, 1] = rows[3][0][0][399].bfloat16().cuda() * 30, -rows[3][0][0][0].bfloat16().cuda() * 30
    got = kvo.paged_attn(q, kp, vp, table, i32(lens), k_scale=ks, v_scale=vs)
    check_attention(q, got, rows, 1, ref.F16)
    kp.view(torch.uint8)[int(table[4, 1]), 0, 3, 5] = 0x7F
    o, lse = kvo.paged_attn(q, kp, vp, table, i32(lens), k_scale=ks, v_scale=vs)
    assert o[4].isnan().all() and lse[4].isnan().all()
    assert torch.equal(o[:4], got[0][:4])


def test_paged_attention_reports_what_is_out_of_range():
    g = gen(2)
    (kp, vp), (ks, vs), table, rows = cache_of(g, [64, 64], 1, 16, 64, True)
    q = normal(g, 2, 4, 64)
    run = lambda tb, ln, **kw: kvo.paged_attn(q, kp, vp, tb, ln, k_scale=ks, v_scale=vs, status=status, **kw)
    good = kvo.paged_attn(q, kp, vp, table, i32([64, 64]), k_scale=ks, v_scale=vs)
    for bad_id in (-1, kp.shape[0], 2 ** 31 - 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tb = table.clone()
        tb[1, 2] = bad_id
        o, _ = run(tb, i32([64, 64]))
        assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID
        assert torch.equal(o[0], good[0][0])
        keep = torch.tensor([t for t in range(64) if t // 16 != 2])
        check_attention(q[1:], (o[1:], _[1:]), [[rows[1][0][:, keep], rows[1][1][:, keep]]], 1, ref.F16)
    for lens in ([64, -3], [64, 10 ** 6]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, _ = run(table, i32(lens))
        assert int(status.item()) == kvo.DEV_BAD_COUNT and torch.equal(o[0], good[0][0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(table, i32([64, 64]), blocks=i32([[[0, 1, -1, 99]], [[0, 1, 2, 3]]]))
    assert int(status.item()) == kvo.DEV_BAD_BLOCK_ID


def test_append_then_attend_step_by_step():
    """Prompts, then tokens one by one, through the 8-bit cache: what a decode loop does, replayed from a graph and
    on a stream of its own."""
    g = gen(21)
    d, hkv, r, page, prompt, steps = 128, 2, 4, 16, [37, 5, 16], 20
    b = len(prompt)
    cap = (max(prompt) + steps + page - 1) // page
    table = torch.randperm(b * cap, generator=g).int().view(b, cap).cuda()
    kp = torch.zeros(b * cap, hkv, page, d, dtype=E4M3, device="cuda")
    vp, ks = torch.zeros_like(kp), torch.ones(b * cap, hkv, device="cuda")
    vs = torch.ones_like(ks)
    freq, amp = kvo.rope_frequencies(d, 500000.0, "banded", 8.0)
    cu = [0]
    for n in prompt:
        cu.append(cu[-1] + n)
    k, v = normal(g, cu[-1], hkv, d), normal(g, cu[-1], hkv, d)
    kvo.paged_append(k, v, kp, vp, table, i32([0] * b), cu=i32(cu), k_scale=ks, v_scale=vs, freq=freq, amplitude=amp)
    lens, start = i32([n + 1 for n in prompt]), i32(prompt)
    q, kn, vn = normal(g, b, hkv * r, d), normal(g, b, hkv, d), normal(g, b, hkv, d)

    def step():
        qr = kvo.paged_append(kn, vn, kp, vp, table, start, k_scale=ks, v_scale=vs, freq=freq, amplitude=amp, q=q)
        out = kvo.paged_attn(qr, kp, vp, table, lens, k_scale=ks, v_scale=vs)
        start.add_(1)
        lens.add_(1)
        return qr, out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qr, got = step()
        for i in range(steps - 1):
            for t in (q, kn, vn):
                t.copy_(normal(g, *t.shape, scale=1.0 + i))
            graph.replay()
            if i % 6 == 5:
                side.synchronize()
                n = [p + 2 + i for p in prompt]
                codes = [(p.double() * s.double()[..., None, None]).cpu() for p, s in ((kp, ks), (vp, vs))]
                rows = [[c[table[j].cpu().long()].transpose(0, 1).flatten(1, 2)[:, :n[j]] for c in codes]
                        for j in range(b)]
                check_attention(qr, got, rows, hkv, ref.F16)
    torch.cuda.current_stream().wait_stream(side)


# ------------------------------------------------------------------ where memory lies, and on which stream
def test_rows_behind_the_last_request_keep_their_bytes():
    g = gen(8)
    kp, vp, ks, vs = pools(g, 4, 1, 16, 64, True)
    k = normal(g, 9, 1, 64)
    q_out, k_out = (torch.full((9, n, 64), 5.0, dtype=torch.bfloat16, device="cuda") for n in (3, 1))
    kvo.paged_append(k, k, kp, vp, i32([[0], [1]]), i32([0, 2]), cu=i32([1, 4, 7]), k_scale=ks, v_scale=vs,
                     freq=kvo.rope_frequencies(64)[0], q=normal(g, 9, 3, 64), q_out=q_out, k_out=k_out)
    for t in (q_out, k_out):
        assert (t[0] == 5.0).all() and (t[7:] == 5.0).all() and (t[1:7] != 5.0).any()


def test_pools_past_four_gigabytes():
    """Pages whose first byte lies past 2^32, rows past 2^31 values: append and attention reach them."""
    g = gen(12)
    hkv, page, d = 2, 128, 128
    n_pages = 2 ** 32 // (hkv * page * d) + 40
    kp, vp = (torch.empty(n_pages, hkv, page, d, dtype=E4M3, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(n_pages, hkv, device="cuda") for _ in range(2))
    table = (n_pages - 1 - torch.arange(6, dtype=torch.int32)).view(2, 3).cuda()
    counts, cu = [300, 129], [0, 300, 429]
    k, v = normal(g, 429, hkv, d), normal(g, 429, hkv, d)
    kvo.paged_append(k, v, kp, vp, table, i32([0, 0]), cu=i32(cu), k_scale=ks, v_scale=vs)
    q = normal(g, 2, 4 * hkv, d)
    got = kvo.paged_attn(q, kp, vp, table, i32(counts), k_scale=ks, v_scale=vs)
    rows = []
    for b, n in enumerate(counts):
        at = table[b].long()
        rows.append([(p[at].float().double() * s[at].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n].cpu()
                     for p, s in ((kp, ks), (vp, vs))])
    for (a, b), (x, y) in zip(((0, 300), (300, 429)), rows):         # the codes are those of the rows appended
        assert ((x.transpose(0, 1) - k[a:b].double().cpu()).abs() <= 2.0 ** -4 * k[a:b].double().cpu().abs() + 2.0 ** -9).all()
    check_attention(q, got, rows, hkv, ref.F16)


def test_calls_on_a_stream_of_their_own():
    """Given a stream, outputs and workspace come from its pool: memory that the current stream frees and takes again
    meanwhile is not touched."""
    g = gen(17)
    lens = [30000, 20000]
    (kp, vp), (ks, vs), table, _ = cache_of(g, lens, 1, 64, 128, True)
    wide = torch.zeros(2, 8192, dtype=torch.int32, device="cuda")          # cut into ranges: a workspace is needed
    wide[:, :table.shape[1]] = table
    q, ln = normal(g, 2, 8, 128), i32(lens)
    want = kvo.paged_attn(q, kp, vp, wide, ln, k_scale=ks, v_scale=vs)
    x = normal(g, 4000, 8, 128)
    pos, (freq, amp) = torch.arange(4000, dtype=torch.int32, device="cuda"), kvo.rope_frequencies(128)
    want_x = kvo.rope(x, pos, freq, amplitude=amp)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        outs = []
        for _ in range(20):
            outs.append((kvo.paged_attn(q, kp, vp, wide, ln, k_scale=ks, v_scale=vs, stream=handle),
                         kvo.rope(x, pos, freq, amplitude=amp, stream=handle)))
            for n in (1 << 12, 1 << 20, 8 << 20):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")    # freed at once
        torch.cuda.synchronize()
        for (o, lse), y in outs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(y, want_x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_no_requests(dtype):
    """An empty batch: empty results, the pools as they were."""
    fp8 = dtype == E4M3
    kp, vp = (torch.zeros(3, 2, 16, 64, device="cuda").to(dtype) for _ in range(2))
    sc = torch.full((3, 2), 0.5, device="cuda") if fp8 else None
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, start = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    status = i32([0])
    q_out = kvo.paged_append(none, none, kp, vp, table, start, k_scale=sc, v_scale=sc, q=q, status=status)
    o, lse = kvo.paged_attn(q, kp, vp, table, start, k_scale=sc, v_scale=sc, status=status)
    assert q_out.shape == o.shape == (0, 8, 64) and lse.shape == (0, 8) and int(status) == 0
    assert not kp.view(torch.uint8).any() and not vp.view(torch.uint8).any()
    o, lse = kvo.prompt_attn(q, none, none, i32([0]), status=status)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8) and int(status) == 0


def test_append_in_place_on_both_paths():
    """k_out is k and q_out is q, contiguous, for one token each and for packed prompts."""
    g = gen(77)
    freq, amp = kvo.rope_frequencies(128)
    for cu, start in ((None, [3, 20, 0]), ([0, 1, 1, 3], [3, 20, 0])):
        k, v, q = normal(g, 3, 2, 128), normal(g, 3, 2, 128), normal(g, 3, 8, 128)
        kw = dict(freq=freq, amplitude=amp, cu=None if cu is None else i32(cu))
        table = i32([[0, 1], [2, 3], [4, 5]])
        pools = [torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        k_out = torch.empty_like(k)
        q_out = kvo.paged_append(k, v, pools[0], pools[1], table, i32(start), q=q, k_out=k_out, **kw)
        k2, q2 = k.clone(), q.clone()
        assert kvo.paged_append(k2, v, pools[2], pools[3], table, i32(start), q=q2, q_out=q2, k_out=k2, **kw) is q2
        assert torch.equal(k2, k_out) and torch.equal(q2, q_out)
        assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_rope_into_views():
    """out apart from x: other heads of the same projection, heads side by side with x's, with other head strides, head
    after head, with padding between tokens."""
    g = gen(6)
    T, H, d = 9, 3, 64
    freq, amp = kvo.rope_frequencies(d)
    pos = i32([5 * i for i in range(T)])
    x = normal(g, T, H, d)
    want = kvo.rope(x, pos, freq)

    def views():
        wide = normal(g, T, 20, d)
        yield wide, wide[:, :H], wide[:, H:2 * H]                              # the next heads
        yield wide, wide[:, 7:7 + H], wide[:, 2:2 + H]                         # heads before
        pairs = wide.view(T, 10, 2, d)
        yield wide, pairs[:, :H, 0], pairs[:, :H, 1]                           # every other head
        yield wide, wide[:, :H], wide[:, 10:10 + 2 * H:2]                      # another head stride
        yield wide, wide[:, 10:10 + 2 * H:2], wide[:, :H]
        planes = normal(g, 2, H, T, d)
        yield planes, planes[0].transpose(0, 1), planes[1].transpose(0, 1)     # head after head
        mixed = normal(g, H, 2, T, d)
        yield mixed, mixed[:, 0].transpose(0, 1), mixed[:, 1].transpose(0, 1)
        rows = normal(g, 2 * T, H, d)
        yield rows, rows[::2], rows[1::2]                                      # every other row
        yield rows, rows[:T], rows[T:]

    for whole, a, b in views():
        a.copy_(x)
        expect = whole.clone()
        at = b.storage_offset(), b.stride()
        expect.as_strided(b.shape, at[1], at[0]).copy_(want)
        kvo.rope(a, pos, freq, out=b)
        assert torch.equal(whole, expect)


def test_outputs_over_what_a_call_reads_are_refused():
    """Views that share memory, from Python: nothing is launched, the buffers keep their bytes."""
    g = gen(4)
    kp, vp, _, _ = pools(g, 8, 2, 16, 64, False)
    kp[0] = 1.0
    k, v, q = normal(g, 2, 2, 64), normal(g, 2, 2, 64), normal(g, 2, 8, 64)
    table, lens = i32([[0, 1], [2, 3]]), i32([20, 9])
    before = kp.clone()
    for call, what in ((lambda: kvo.paged_append(k, v, kp, kp, table, lens), "of their own"),
                       (lambda: kvo.paged_append(k, v, kp, vp, table, lens, k_out=kp.view(-1)[:256].view(2, 2, 64)), "nothing else"),
                       (lambda: kvo.paged_attn(q, kp, vp, table, lens, o=kp.view(-1)[:1024].view(2, 8, 64)), "apart"),
                       (lambda: kvo.paged_attn(q, kp, vp, table, lens, lse=q.view(-1).view(torch.float32)[:16].view(2, 8)), "apart"),
                       (lambda: kvo.prompt_attn(q, k, v, i32([0, 2]), lse=k.view(-1).view(torch.float32)[:16].view(2, 8)), "apart")):
        with pytest.raises(kvo.KvoError, match=what):
            call()
    assert torch.equal(kp, before)
    # K and V read from one pool are no output
    o, lse = kvo.paged_attn(q, kp, kp, table, lens)
    check_attention(q, (o, lse), [[kp[i32([2 * b, 2 * b + 1]).long()].double().cpu().transpose(0, 1).flatten(1, 2)[:, :n]] * 2
                                  for b, n in enumerate([20, 9])], 2, ref.BF16)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("cap,lens", [(8000, [3000, 0, 700]), (60, [900, 70, 1])])     # ranges, clusters
def test_paged_attention_into_given_buffers(e4m3, cap, lens):
    """The caller's o, lse and workspace, whatever they and the memory behind them hold; a workspace too small is refused."""
    g = gen(cap)
    (kp, vp), (ks, vs), table, rows = cache_of(g, lens, 2, 16, 128, e4m3)
    wide = torch.zeros(len(lens), cap, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = normal(g, len(lens), 8, 128)
    kw = dict(k_scale=ks, v_scale=vs)
    want = kvo.paged_attn(q, kp, vp, wide, i32(lens), **kw)
    check_attention(q, want, rows, 2, ref.F16 if e4m3 else ref.BF16)
    space = torch.full((32 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    for fill in (0xFF, 0x7F, 0):
        space.fill_(fill)
        o, lse = torch.full_like(q, math.nan), torch.full((len(lens) + 1, 8), 3.0, device="cuda")
        got = kvo.paged_attn(q, kp, vp, wide, i32(lens), o=o, lse=lse[:-1], workspace=space, **kw)
        assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == lse.data_ptr()
        assert torch.equal(o, want[0]) and torch.equal(lse[:-1], want[1]) and bool((lse[-1] == 3.0).all())
    if cap == 8000:
        with pytest.raises(kvo.KvoError, match="too small"):
            kvo.paged_attn(q, kp, vp, wide, i32(lens), workspace=space[:1024], **kw)
