"""A paged cache as a server runs it, every step through the calls that belong to it: prompts in chunks, samples that share
a prompt's pages, drafts that are verified and cut back, requests that end, pages moved together, single tokens.  Each
attention is compared with a plain 64-bit one over what the pages hold, and what they hold with the tokens that went in."""
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


class Server:
    LAYERS = 2

    def __init__(self, seed, batch, hkv, r, d, page, n_pages, width, e4m3, stream):
        self.g, self.rng = torch.Generator().manual_seed(seed), random.Random(seed)
        self.batch, self.hkv, self.r, self.d, self.page, self.n_pages, self.e4m3 = batch, hkv, r, d, page, n_pages, e4m3
        shape = (self.LAYERS, n_pages, hkv, page, d)
        # codes and scales that were never written are NaN
        self.k, self.v = (torch.full(shape, float("nan")).to(E4M3 if e4m3 else torch.bfloat16).cuda() for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:3], float("nan"), device="cuda") if e4m3 else None for _ in range(2))
        self.table, self.held, self.refs = i32([[-1] * width] * batch), i32([0] * batch), i32([0] * n_pages)
        self.tokens = [[] for _ in range(batch)]             # of each request: per token (k, v) [layers][hkv][d]
        self.status, self.stream = i32([0]), stream

    def scales(self, layer):
        return dict(k_scale=self.ks[layer], v_scale=self.vs[layer]) if self.e4m3 else {}

    def lens(self):
        return [len(t) for t in self.tokens]

    def book(self):
        """Each page is named as often as refs says; a page that is written next belongs to one request."""
        table, held, refs = self.table.tolist(), self.held.tolist(), self.refs.tolist()
        uses = [0] * self.n_pages
        for row, n, t in zip(table, held, self.tokens):
            assert n * self.page >= len(t) and all(p == -1 for p in row[n:])
            for p in row[:n]:
                uses[p] += 1
        assert uses == refs
        for row, t in zip(table, self.tokens):
            if len(t) % self.page:
                assert refs[row[len(t) // self.page]] == 1
        assert int(self.status.item()) == 0

    def add(self, new, q_rows=True):
        """new[b] tokens for each request, and their attention, layer by layer."""
        start, cu = self.lens(), cuts(new)
        kv = torch.randn(2, self.LAYERS, cu[-1], self.hkv, self.d, generator=self.g).bfloat16()
        q = torch.randn(self.LAYERS, cu[-1], self.hkv * self.r, self.d, generator=self.g).bfloat16().cuda()
        for b, n in enumerate(new):
            self.tokens[b] += [(kv[0, :, cu[b] + i], kv[1, :, cu[b] + i]) for i in range(n)]
        kv, s = kv.cuda(), dict(status=self.status, stream=self.stream)
        torch.cuda.synchronize()
        kvo.paged_reserve(self.table, self.held, self.refs, i32(self.lens()), self.page, **s)
        outs = []
        lens, cu, first = i32(self.lens()), i32(cu), i32(start)
        for x in range(self.LAYERS):
            kvo.paged_append(kv[0, x], kv[1, x], self.k[x], self.v[x], self.table, first, cu=cu, **self.scales(x), **s)
            o, lse = kvo.paged_chunk_attn(q[x], self.k[x], self.v[x], self.table, lens, cu, max_new=max(new), max_len=max(self.lens()),
                                          **self.scales(x), **s)
            outs.append((o, lse))
            if all(n == 1 for n in new):
                one = kvo.paged_attn(q[x], self.k[x], self.v[x], self.table, lens, **self.scales(x), **s)
                outs.append(one)
        torch.cuda.synchronize()
        self.book()
        self.holds()
        for i, (o, lse) in enumerate(outs):
            x = i * self.LAYERS // len(outs)
            self.attended(x, q[x].cpu(), new, o, lse)
        return q, cu, outs

    def rows(self, x, b):
        """(k, v) [n][hkv][d] in 64 bits of what layer x's pages hold of request b, and the scale of each value."""
        n, out = len(self.tokens[b]), []
        ids = self.table[b, :-(-n // self.page)].long()
        for pool, scale in ((self.k, self.ks), (self.v, self.vs)):
            y = pool[x, ids].double().cpu().transpose(1, 2).reshape(-1, self.hkv, self.d)
            s = torch.zeros_like(y)
            if self.e4m3:
                s = scale[x, ids].double().cpu()[:, None, :, None].expand(-1, self.page, -1, self.d).reshape(-1, self.hkv, self.d)
                y = y * s
            out += [y[:n], s[:n]]
        return out

    def holds(self):
        for b, t in enumerate(self.tokens):
            for x in range(self.LAYERS if t else 0):
                k, ks, v, vs = self.rows(x, b)
                for i, (got, s) in enumerate(((k, ks), (v, vs))):
                    want = torch.stack([y[i][x] for y in t]).double()
                    # e4m3: half a step of a value, or of the smallest (2^-10 of the scale), and as much again for all the
                    # scales below it that a page had before, each at most half of the next
                    tol = 2.0 ** -4 * want.abs() + 2.0 ** -9 * s if self.e4m3 else torch.zeros_like(want)
                    assert bool(((got - want).abs() <= tol).all()), (b, x, i)

    def attended(self, x, q, new, o, lse):
        cu = cuts(new)
        for b, n in enumerate(new):
            if n == 0:
                continue
            k, _, v, _ = self.rows(x, b)
            have = len(self.tokens[b])
            for i in sorted({0, n - 1, self.rng.randrange(n)}):
                for h in (0, self.hkv * self.r - 1):
                    see, g, row = have - n + i + 1, h // self.r, q[cu[b] + i, h].double()
                    want, wl, tol, tl = ref.attention(row, k[:see, g], v[:see, g], 2 * ref.BF16 if self.e4m3 else ref.BF16)
                    if self.e4m3:          # q as two e4m3 values, each within 2^-17 of the row's largest
                        ds = float(2.0 ** -17 * row.abs().max() * k[:see, g].abs().sum(1).max() / self.d ** 0.5)
                        tol, tl = tol + 2 * ds * (torch.softmax(k[:see, g] @ row / self.d ** 0.5, 0) @ v[:see, g].abs()), tl + ds
                    ref.check(o[cu[b] + i, h], want, tol, f"o of request {b}, token {i}, head {h}")
                    assert abs(float(lse[cu[b] + i, h]) - wl) <= tl

    def fork(self, parent, keep):
        s = dict(status=self.status, stream=self.stream)
        torch.cuda.synchronize()
        moves = kvo.paged_fork(self.table, self.held, self.refs, i32(parent), i32(keep), self.page, **s)
        kvo.paged_copy(self.k, self.v, *moves, k_scale=self.ks, v_scale=self.vs, **s)
        torch.cuda.synchronize()
        self.tokens = [list(self.tokens[p][:n]) if p >= 0 else [] for p, n in zip(parent, keep)]
        self.book()
        self.holds()
        return int(moves[2].item())

    def compact(self):
        s = dict(status=self.status, stream=self.stream)
        torch.cuda.synchronize()
        moves = kvo.paged_compact(self.table, self.held, self.refs, **s)
        kvo.paged_copy(self.k, self.v, *moves, k_scale=self.ks, v_scale=self.vs, **s)
        torch.cuda.synchronize()
        self.book()
        self.holds()
        used = sum(r > 0 for r in self.refs.tolist())
        assert all(r > 0 for r in self.refs.tolist()[:used])
        return int(moves[2].item())


@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,r,d,page", [(2, 4, 128, 16), (1, 3, 64, 32)])
def test_a_server(hkv, r, d, page, e4m3, own_stream):
    s = Server(7, 9, hkv, r, d, page, 130, 24, e4m3, torch.cuda.Stream() if own_stream else None)
    s.add([70, 33, 1, 0, 129, 0, 0, 0, 16])              # prompts, one of them in two chunks
    s.add([0, 1, 40, 0, 100, 0, 0, 0, 1])
    lens = s.lens()
    # Requests 5 to 7 are samples of 0 and 4: part-filled pages are copied, whole ones shared.
    assert s.fork([0, 1, 2, -1, 4, 0, 4, 4, 8], [lens[0], lens[1], lens[2], 0, lens[4], lens[0], lens[4], page * 3 + 1, lens[8]]) > 0
    for round_ in range(3):                              # drafts of up to four tokens, of which some are kept
        draft = [s.rng.randint(1, 4) if s.tokens[b] else 0 for b in range(9)]
        before = s.lens()
        s.add(draft)
        s.fork(list(range(9)), [n + s.rng.randint(0, m) for n, m in zip(before, draft)])
    lens = s.lens()
    s.fork([0, 6, -1, 5, 4, 5, -1, 7, 0], [lens[0], lens[6], 0, 30, lens[4], lens[5], 0, lens[7], lens[0]])       # beams reordered, two ended
    # Behind the move attention gives the same bits.
    lens, live = s.lens(), [b for b in range(9) if s.tokens[b]]
    new = [min(3, n) for n in lens]
    q = torch.randn(sum(new), hkv * r, d, generator=s.g).bfloat16().cuda()
    call = lambda: [kvo.paged_chunk_attn(q, s.k[x], s.v[x], s.table, i32(lens), i32(cuts(new)), max_new=m, status=s.status, **s.scales(x))
                    for x in range(s.LAYERS) for m in (0, 3)]
    want = call()
    assert s.compact() > 0 and live
    for a, b in zip(want, call()):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s.add([1] * 9)                                       # single tokens, for requests that were empty too
    s.add([20, 1, 50, 3, 1, 1, 7, 1, 1])
    s.fork([-1] * 9, [0] * 9)
    assert not s.refs.any()
