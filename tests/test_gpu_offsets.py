"""Bad offsets of packed requests: a request whose offsets descend, leave the tokens or begin before the end of an earlier
one is skipped and reported, and in calls of up to 32 requests every row of every other request is there."""
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


def many(changes, n, each=50):
    cu = [each * i for i in range(n + 1)]
    for i, x in changes.items():
        cu[i] = x
    return cu, [cu[i + 1] if changes.keys() & {i} else cu[i] for i in range(n + 1)]


# offsets, ascending offsets with the same served requests, and those requests
SOME = {
    "negative": ([0, 3200, -4, 6400], [0, 3200, 3200, 6400], [0]),
    "small": ([0, 3200, 10, 20, 6400], [0, 3200, 3200, 3200, 6400], [0]),
    "past the end": ([0, 300, 9000, 400, 6400], [0, 300, 400, 400, 6400], [0, 3]),
    "overlap": ([0, 3200, 10, 3300, 6400], [0, 3200, 3200, 3300, 6400], [0, 3]),
    "first": ([50, 20, 3000, 6400], [20, 20, 3000, 6400], [1, 2]),
    "last": ([0, 100, 3200, 6401], [0, 100, 3200, 6400], [0, 1]),
}
MANY = {
    "32, negative": (*many({20: -4}, n=32), [i for i in range(32) if i not in (19, 20)]),
    "32, past": (*many({3: 99999}, n=32), [i for i in range(32) if i not in (2, 3)]),
    "32, small": (*many({25: 7, 12: -1}, n=32), [i for i in range(32) if i not in (11, 12, 24, 25)]),
}
CASES = [pytest.param(*v, id=k) for k, v in {**SOME, **MANY}.items()]


def rows_of(cu, served, total):
    keep = torch.zeros(total, dtype=torch.bool)
    for b in served:
        keep[cu[b]:cu[b + 1]] = True
    return keep.cuda()


@pytest.mark.parametrize("bad,good,served", CASES)
@pytest.mark.parametrize("d,hkv,r", [(64, 1, 4), (128, 2, 3)])
def test_prompt_attention_serves_the_other_requests(d, hkv, r, bad, good, served):
    g = gen(len(bad))
    T = good[-1]
    q, k, v = normal(g, T, hkv * r, d), normal(g, T, hkv, d), normal(g, T, hkv, d)
    want = kvo.prompt_attn(q, k, v, i32(good))
    o, lse = torch.full_like(q, 7.0), torch.full((T, hkv * r), 7.0, device="cuda")
    status = i32([0])
    kvo.prompt_attn(q, k, v, i32(bad), o=o, lse=lse, status=status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    keep = rows_of(good, served, T)
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert bool((o[~keep] == 7.0).all()) and bool((lse[~keep] == 7.0).all())
    # bad offsets of the keys alone
    o.fill_(7.0)
    kvo.prompt_attn(q, k, v, i32(good), i32(good[:-1] + [T + 1]), o=o)
    last = rows_of(good, range(len(good) - 2), T)
    assert torch.equal(o[last], want[0][last]) and bool((o[~last] == 7.0).all())


@pytest.mark.parametrize("bad,good,served", CASES)
@pytest.mark.parametrize("e4m3,page,d,hkv", [(True, 16, 64, 1), (False, 64, 128, 2), (True, 32, 128, 8)])
def test_append_serves_the_other_requests(e4m3, page, d, hkv, bad, good, served):
    g = gen(len(bad) + page)
    T, b, hq = good[-1], len(good) - 1, 4 * hkv
    start = [(7 * i) % (2 * page) for i in range(b)]
    per = max((s + good[i + 1] - good[i] + page - 1) // page for i, s in enumerate(start)) + 1
    table = torch.randperm(b * per, generator=g).int().view(b, per).cuda()
    q, k, v = normal(g, T, hq, d), normal(g, T, hkv, d), normal(g, T, hkv, d)
    freq = kvo.rope_frequencies(d)[0]

    def run(cu, status=None):
        pools = [torch.zeros(b * per, hkv, page, d, device="cuda").to(E4M3 if e4m3 else torch.bfloat16) for _ in range(2)]
        scale = [torch.ones(b * per, hkv, device="cuda") if e4m3 else None for _ in range(2)]
        q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        kvo.paged_append(k, v, *pools, table, i32(start), cu=i32(cu), k_scale=scale[0], v_scale=scale[1], freq=freq, q=q,
                         q_out=q_out, k_out=k_out, status=status)
        return [t.view(torch.uint8) for t in pools] + [s for s in scale if e4m3], (q_out, k_out)

    status = i32([0])
    want, want_rows = run(good)
    got, got_rows = run(bad, status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    keep = rows_of(good, served, T)
    for x, y in zip(got_rows, want_rows):
        assert torch.equal(x[keep], y[keep]) and bool((x[~keep] == 7.0).all())
    mine = torch.zeros(b * per, dtype=torch.bool, device="cuda")
    mine[table[list(served)].long().flatten()] = True
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[mine], y[mine])
        assert bool((x[~mine] == (0 if i < 2 else 1)).all())


def test_bad_offsets_among_many_requests():
    """More than 32: reported, and a row is as it should be or as it was."""
    bad, good = many({20: -4}, n=40)
    served = [i for i in range(40) if i not in (19, 20)]
    g = gen(1)
    T = good[-1]
    q, k, v = normal(g, T, 4, 64), normal(g, T, 1, 64), normal(g, T, 1, 64)
    want, _ = kvo.prompt_attn(q, k, v, i32(good))
    o, status = torch.full_like(q, 7.0), i32([0])
    kvo.prompt_attn(q, k, v, i32(bad), o=o, status=status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    keep = rows_of(good, served, T)
    same, left = (o == want).flatten(1).all(1), (o == 7.0).flatten(1).all(1)
    assert bool((same | left)[keep].all()) and bool(left[~keep].all())
    table = torch.arange(40 * 4, dtype=torch.int32, device="cuda").view(40, 4)
    pool = lambda: [torch.zeros(160, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    one, two = pool(), pool()
    kvo.paged_append(k, v, *one, table, i32([0] * 40), cu=i32(good))
    status.zero_()
    kvo.paged_append(k, v, *two, table, i32([0] * 40), cu=i32(bad), status=status)
    assert int(status.item()) == kvo.DEV_BAD_COUNT
    for x, y in zip(one, two):
        assert bool(((x == y).flatten(1).all(1) | (y == 0).flatten(1).all(1)).all())
