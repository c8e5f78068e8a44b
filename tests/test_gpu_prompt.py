"""Attention over packed prompts against a plain 64-bit reference, and the way from a prompt to decode steps."""
import math

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()


def cuts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_rows(q, k, v, o, lse, cq, ck, causal, rows=None):
    """Rows (token, head) of the packed call, each against the 64-bit attention of its own request."""
    hq, r = q.shape[1], q.shape[1] // k.shape[1]
    kd, vd = k.double().cpu(), v.double().cpu()
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for i in range(nq) if rows is None else [x for x in rows if x < nq]:
            see = min(max(i + 1 + nk - nq, 0), nk) if causal else nk
            for h in range(hq):
                want, wl, tol, tl = ref.attention(q[cq[b] + i, h].double().cpu(), kd[ck[b]:ck[b] + see, h // r],
                                                  vd[ck[b]:ck[b] + see, h // r], ref.BF16)
                ref.check(o[cq[b] + i, h], want, tol, f"o of request {b}, token {i}, head {h}")
                got = float(lse[cq[b] + i, h])
                assert got == wl or abs(got - wl) <= tl, (b, i, h, got, wl)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,hkv,r,nq,nk", [
    (128, 1, 1, [1], None), (64, 1, 1, [1], None), (128, 1, 4, [130], None), (64, 2, 4, [3, 0, 129, 1, 64], None),
    (128, 2, 1, [257], None), (64, 1, 16, [40, 9], None), (128, 1, 3, [50, 200], None), (128, 1, 7, [91], None),
    (64, 1, 12, [33, 1], None), (128, 2, 2, [5, 1, 70], [300, 128, 70]), (64, 1, 5, [20, 30, 4], [7, 0, 129]),
    (128, 1, 8, [1, 1, 1], [500, 1, 255])])
def test_prompt_attention_matches_reference(causal, d, hkv, r, nq, nk):
    g = gen(sum(nq) + r)
    cq, ck = cuts(nq), cuts(nk or nq)
    q = normal(g, cq[-1], hkv * r, d, scale=1.5)
    k, v = normal(g, ck[-1], hkv, d), normal(g, ck[-1], hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kvo.prompt_attn(q, k, v, i32(cq), None if nk is None else i32(ck), causal, status=status)
    assert int(status.item()) == 0
    check_rows(q, k, v, o, lse, cq, ck, causal)
    again = kvo.prompt_attn(q, k, v, i32(cq), i32(ck), causal)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("d,r,n,scale", [(128, 4, 2500, 1.0), (64, 2, 4100, 6.0), (128, 1, 1300, 20.0)])
def test_prompt_attention_long(d, r, n, scale):
    """Long prompts, with scores that spread far enough for the running maximum to rise late."""
    g = gen(n)
    q, k, v = normal(g, n, r, d, scale=scale), normal(g, n, 1, d), normal(g, n, 1, d)
    o, lse = kvo.prompt_attn(q, k, v, i32([0, n]))
    check_rows(q, k, v, o, lse, [0, n], [0, n], True, rows=[0, 1, 127, 128, 129, 255, 256, 640, n // 2, n - 2, n - 1])


@pytest.mark.parametrize("d,hkv,r", [(128, 8, 4), (64, 16, 2)])
def test_prompt_attention_fills_the_device(d, hkv, r):
    """Enough items that each has a CTA of its own."""
    g = gen(d)
    n = 1300
    q, k, v = normal(g, n, hkv * r, d, scale=3.0), normal(g, n, hkv, d), normal(g, n, hkv, d)
    o, lse = kvo.prompt_attn(q, k, v, i32([0, n]))
    check_rows(q, k, v, o, lse, [0, n], [0, n], True, rows=[0, 127, 128, 700, n - 1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,hkv,r,nq,nk", [
    (128, 1, 4, [5], [1500]), (64, 1, 1, [1], [2000]), (128, 2, 3, [50], [1153]), (64, 1, 16, [3], [1024]),
    (128, 1, 2, [5, 0, 40], [3000, 700, 17]), (64, 2, 5, [1, 9, 300], [4000, 1, 260]), (128, 8, 4, [200], [1500]),
    (64, 8, 4, [130, 60], [2500, 900]), (128, 8, 4, [500], [2000]), (64, 4, 8, [300], [2100])])
def test_prompt_attention_splits_long_keys(causal, d, hkv, r, nq, nk):
    """Few query rows and many keys: a cluster shares each item's keys.  Parts without a tile, requests that end within
    the first part, rows that see nothing, and NaN behind the last key."""
    g = gen(sum(nk) + r)
    cq, ck = cuts(nq), cuts(nk)
    q, k, v = (normal(g, n, h, d, scale=s) for n, h, s in ((cq[-1], hkv * r, 2.0), (ck[-1] + 40, hkv, 1.0), (ck[-1] + 40, hkv, 1.0)))
    k[ck[-1]:], v[ck[-1]:] = math.nan, math.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kvo.prompt_attn(q, k, v, i32(cq), i32(ck), causal, status=status)
    assert int(status.item()) == 0
    check_rows(q, k, v, o, lse, cq, ck, causal, rows=[0, 1, 4, 30, 39, 63, 64, 129, 199, 299, 499])
    again = kvo.prompt_attn(q, k, v, i32(cq), i32(ck), causal)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_prompt_attention_split_ignores_other_requests():
    """A request of NaN keys and values and one with bad offsets beside one whose keys are split."""
    g = gen(61)
    q, k, v = normal(g, 30, 4, 128), normal(g, 5000, 1, 128), normal(g, 5000, 1, 128)
    k[2300:], v[2300:] = math.nan, math.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((30, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((30, 4), 7.0, device="cuda")
    kvo.prompt_attn(q, k, v, i32([0, 10, 15, 20]), i32([0, 2300, 4000, 5001]), o=o, lse=lse, status=status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    check_rows(q, k, v, o, lse, [0, 10], [0, 2300], True)
    assert bool(o[10:15].isnan().all()) and bool((o[15:] == 7.0).all()) and bool((lse[15:] == 7.0).all())


def test_prompt_attention_keeps_requests_apart():
    """Views of a fused projection with NaN in the padding and in a neighbour: other requests' rows stay clean, and
    rows behind the last request keep their bytes."""
    g = gen(9)
    hq, hkv, d = 8, 2, 128
    nq = [70, 30, 200]
    cq = cuts(nq)
    qkv = normal(g, cq[-1] + 40, hq + 2 * hkv, d)
    qkv[cq[-1]:] = math.nan
    want = qkv.clone()
    qkv[cq[1]:cq[2]] = math.nan
    o = torch.full((cq[-1] + 40, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cq[-1] + 40, hq), 3.0, device="cuda")
    for causal in (True, False):
        kvo.prompt_attn(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], i32(cq), causal=causal, o=o, lse=lse)
        assert (o[cq[-1]:] == 3.0).all() and (lse[cq[-1]:] == 3.0).all()
        assert o[cq[1]:cq[2]].isnan().all()
        for b in (0, 2):
            sl = slice(cq[b], cq[b + 1])
            alone = kvo.prompt_attn(*(want[sl, a:e] for a, e in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))),
                                    i32([0, nq[b]]), causal=causal)
            assert torch.equal(o[sl], alone[0]) and torch.equal(lse[sl], alone[1])


def test_prompt_attention_reports_bad_offsets():
    g = gen(4)
    q, k, v = normal(g, 40, 2, 64), normal(g, 40, 1, 64), normal(g, 40, 1, 64)
    good = kvo.prompt_attn(q, k, v, i32([0, 10, 40]))
    for cq, ck, ok in (([0, 10, 41], [0, 10, 40], 0), ([0, 10, 40], [0, 10, 900], 0), ([0, 10, 40], [0, 10, 5], 0),
                       ([0, 10, -4], [0, 10, 40], 0)):
        o = torch.full_like(q, 2.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvo.prompt_attn(q, k, v, i32(cq), i32(ck), o=o, status=status)
        assert int(status.item()) == kvo.DEV_BAD_COUNT
        assert torch.equal(o[:10], good[0][:10]) and (o[10:] == 2.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_from_prompt_to_decode(e4m3):
    """A whole run: positions on q and k, attention over the prompts, the cache filled by the same call, then a
    decode step over it -- which must agree with the prompt attention of the prompt one token longer -- and, over
    blocks chosen per KV head, with the offloaded context's own selection and attention."""
    g = gen(31)
    hq, hkv, d, page = 8, 2, 128, 32
    nq = [96 + 32 * 9, 97 + 32 * 7]
    cq, b = cuts(nq), len(nq)
    qkv = normal(g, cq[-1], hq + 2 * hkv, d)
    freq, amp = kvo.rope_frequencies(d, 500000.0)
    cap = (max(nq) + page - 1) // page
    table = torch.randperm(b * cap, generator=g).int().view(b, cap).cuda()
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kp, vp = (torch.zeros(b * cap, hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(b * cap, hkv, device="cuda") for _ in range(2)) if e4m3 else (None, None)
    k_out = torch.empty(cq[-1], hkv, d, dtype=torch.bfloat16, device="cuda")
    q = kvo.paged_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, table, i32([0] * b), cu=i32(cq), k_scale=ks,
                         v_scale=vs, freq=freq, amplitude=amp, q=qkv[:, :hq], k_out=k_out)
    pos = torch.cat([torch.arange(n) for n in nq]).int().cuda()
    both = kvo.rope(qkv[:, :hq + hkv], pos, freq, amplitude=amp)
    assert torch.equal(both[:, :hq], q) and torch.equal(both[:, hq:], k_out)
    o, lse = kvo.prompt_attn(q, k_out, qkv[:, hq + hkv:], i32(cq))
    check_rows(q, k_out, qkv[:, hq + hkv:], o, lse, cq, cq, True, rows=[0, 31, 128, 200, min(nq) - 1])
    # the last token's row again, as a decode step over the cache
    last = torch.tensor([c - 1 for c in cq[1:]], device="cuda")
    o2, lse2 = kvo.paged_attn(q[last].contiguous(), kp, vp, table, i32(nq), k_scale=ks, v_scale=vs)
    if e4m3:      # against the values that the 8-bit cache stands for
        full = [(p.double() * s.double()[..., None, None]).cpu() for p, s in ((kp, ks), (vp, vs))]
    else:
        full = [p.double().cpu() for p in (kp, vp)]
    for i in range(b):
        kk, vv = (f[table[i].cpu().long()].transpose(0, 1).flatten(1, 2)[:, :nq[i]] for f in full)
        for h in range(hq):
            want, wl, tol, tl = ref.attention(q[last[i], h].double().cpu(), kk[h // 4], vv[h // 4],
                                              ref.F16 if e4m3 else ref.BF16)
            ref.check(o2[i, h], want, tol, "decode")
            assert abs(float(lse2[i, h]) - wl) <= tl
    if e4m3:
        return
    # The same keys offloaded: the context's window is the last 32 (and one more) tokens, its blocks the pages before
    i, W, k_sel = 0, 96, 4
    n = nq[i]
    host = [t[cq[i]:cq[i + 1]].transpose(0, 1).contiguous().cpu().pin_memory() for t in (k_out, qkv[:, hq + hkv:])]
    win = [h[:, n - W:].contiguous().cuda().view(1, hkv, W, d) for h in host]
    ctx = kvo.Context(batch=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, block_size=page, top_k=k_sel, window=W,
                      n_layers=1, seq_lens=[n], k_host=[host[0]], v_host=[host[1]], k_win=[win[0]], v_win=[win[1]])
    try:
        q1 = q[last[i]].view(1, hq, d).contiguous()
        T, _ = ctx.select_topk(0, q1)
        want, want_lse = ctx.decode_step(q1.unsqueeze(0))
        tail = torch.arange((n - W) // page, n // page, dtype=torch.int32, device="cuda").expand(hkv, -1)
        blocks = torch.cat([T.view(hkv, k_sel), tail], dim=1).contiguous().view(1, hkv, -1)
        o3, lse3 = kvo.paged_attn(q1, kp, vp, table[i:i + 1], i32([n]), blocks=blocks)
        torch.cuda.synchronize()
        assert (o3.float().view(-1) - want.view(-1)).abs().max() <= 2e-2
        assert (lse3.view(-1) - want_lse.view(-1)).abs().max() <= 1e-3
    finally:
        ctx.close()


def test_prompt_attention_past_four_gigabytes():
    """A request whose rows lie past 2^31 values of q, k, v and o."""
    g = gen(41)
    hq, hkv, d, n = 32, 32, 128, 150
    T = 2 ** 32 // (2 * hq * d) + 5000
    q, k, v = (torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    o = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, hq), 2.0, device="cuda")
    for t in (q, k, v):
        t[T - n:] = normal(g, n, hq, d)
    o[T - n - 64:T - n] = 7.0
    cu = [T - n, T]
    kvo.prompt_attn(q, k, v, i32(cu), o=o, lse=lse)
    check_rows(q[T - n:], k[T - n:], v[T - n:], o[T - n:], lse[T - n:], [0, n], [0, n], True, rows=[0, 77, n - 1])
    assert (o[T - n - 64:T - n] == 7.0).all() and (lse[:T - n] == 2.0).all()


def test_many_requests_in_one_call():
    """More requests than one round of offsets holds, empty ones among them."""
    g = gen(43)
    nq = [(7 * i) % 5 for i in range(90)]
    cq = cuts(nq)
    q, k, v = normal(g, cq[-1], 4, 64), normal(g, cq[-1], 2, 64), normal(g, cq[-1], 2, 64)
    o, lse = kvo.prompt_attn(q, k, v, i32(cq))
    check_rows(q, k, v, o, lse, cq, cq, True)


def test_calls_in_two_graphs_and_streams():
    """Prompt attention, append and decode captured twice and replayed side by side, each with its own outputs."""
    g = gen(47)
    n, hq, hkv, d = 200, 8, 2, 64
    sets = []
    for _ in range(2):
        s = dict(q=normal(g, n, hq, d), k=normal(g, n, hkv, d), v=normal(g, n, hkv, d), cu=i32([0, 77, n]),
                 kp=torch.zeros(64, hkv, 16, d, dtype=torch.bfloat16, device="cuda"), table=torch.arange(32, dtype=torch.int32, device="cuda").view(2, 16))
        s["vp"] = torch.zeros_like(s["kp"])
        sets.append(s)

    def run(s):
        kvo.paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], i32_zero, cu=s["cu"])
        a = kvo.prompt_attn(s["q"], s["k"], s["v"], s["cu"])
        return a + kvo.paged_attn(s["q"][:2].contiguous(), s["kp"], s["vp"], s["table"], lens)

    i32_zero, lens = i32([0, 0]), i32([77, 123])
    want = [[t.clone() for t in run(s)] for s in sets]
    graphs = []
    for s in sets:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            out = run(s)
        graphs.append((gr, st, out))
    torch.cuda.synchronize()
    for _ in range(30):
        for gr, st, _o in graphs:
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for w, (_g, _s, out) in zip(want, graphs):
        for a, b in zip(w, out):
            assert torch.equal(a, b)
