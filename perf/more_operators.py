"""Cases of the operators that keep a paged cache through its life: attention of new tokens over the cached pages (bf16,
or 8 bits with a scale per page and KV head), and the pages' bookkeeping (reserving, forking, freeing, compacting,
copying).

``own`` False computes the plain forms with elementary torch operations in 32 bits; True calls the library.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128}
    return [
        # one request checks three drafted tokens: latency only
        {"name": "chunk_verify_1x4_bf16", "op": "chunk", "hq": 8, "hkv": 2, "d": 64, "batch": 1, "one": 0, "tokens": 4,
         "lo": 4092, "hi": 4092, "page": 16, "bits": 16},
        # 48 requests check three drafted tokens each over long ragged contexts: the cache's bytes
        {"name": "chunk_verify_48x4_e4m3", "op": "chunk", **llama, "batch": 48, "one": 0, "tokens": 192, "lo": 8192,
         "hi": 32768, "page": 32, "bits": 8},
        # a serving step of 36 requests with one token each and four pieces of prompts, odd heads
        {"name": "chunk_mixed_40_bf16", "op": "chunk", "hq": 20, "hkv": 4, "d": 128, "batch": 40, "one": 36,
         "tokens": 1987, "lo": 100, "hi": 9001, "page": 64, "bits": 16},
        # a piece of a long prompt behind 30000 cached tokens: the tensor cores
        {"name": "chunk_2048_behind_30000_e4m3", "op": "chunk", **llama, "batch": 1, "one": 0, "tokens": 2048, "lo": 30000,
         "hi": 30000, "page": 64, "bits": 8},
        # three pages of one layer of a small model (forks of three beams)
        {"name": "copy_3_pages_bf16", "op": "copy", "hkv": 2, "d": 64, "page": 16, "bits": 16, "layers": 1, "pages": 257,
         "moves": 3},
        # what a compaction moves in four layers
        {"name": "copy_501_pages_4_layers_e4m3", "op": "copy", "hkv": 8, "d": 128, "page": 64, "bits": 8, "layers": 4,
         "pages": 2048, "moves": 501},
        # a step of a search with four beams for each of eight prompts
        {"name": "fork_beams_8x4", "op": "fork", "kind": "beams", "batch": 32, "group": 4, "page": 32, "lo": 700,
         "hi": 2100, "pages": 8192},
        # a batch's slots taken over by forks of 32 cached prefixes, the requests that held them ended
        {"name": "fork_prefixes_256", "op": "fork", "kind": "prefixes", "batch": 256, "group": 8, "page": 16, "lo": 2000,
         "hi": 16384, "pages": 196608},
        # rejected drafts given back, room for the next ones taken
        {"name": "reserve_drafts_48", "op": "reserve", "kind": "drafts", "batch": 48, "page": 32, "lo": 8192, "hi": 32768,
         "pages": 65536, "add": 5},
        # ended requests leave, as many new prompts are given their pages
        {"name": "reserve_prompts_192", "op": "reserve", "kind": "prompts", "batch": 192, "page": 16, "lo": 500,
         "hi": 16384, "pages": 262144, "add": 0},
        # a small pool whose requests ended here and there
        {"name": "compact_2048", "op": "compact", "batch": 13, "page": 64, "lo": 1, "hi": 8000, "pages": 2048, "gone": 3},
        # a large one
        {"name": "compact_262144", "op": "compact", "batch": 256, "page": 16, "lo": 1000, "hi": 20000, "pages": 262144,
         "gone": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "copy", "fork", "reserve", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "chunk":
        most = [work(c) for c in listed()]
        most = {x: max(w[x] for w in most) for x in ("bytes", "flops")}
        while True:
            d = rng.choice([64, 128, 128])
            hkv = rng.choice([1, 2, 4, 8])
            hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            batch = _log(rng, 1, 128)
            kind = rng.choice(["verify", "chunks", "mixed"])
            one = 0 if kind != "mixed" else rng.randrange(batch)
            tokens = batch * rng.randint(1, 8) if kind == "verify" else batch + _log(rng, 1, 8000)
            hi = _log(rng, 1, 65536) - 1
            case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "batch": batch, "one": one, "tokens": tokens,
                    "lo": hi // rng.choice([1, 2, 16]), "hi": hi, "page": page, "bits": rng.choice([8, 8, 16])}
            w = work(case)
            n, past = _cuts(case), _pasts(case)
            wide = 4 * batch * hq * max(n) * (max(past) + max(n))       # the plain form's scores, padded
            if hq <= 64 and all(w[x] <= most[x] for x in most) and wide <= 12e9:
                return case
    if op == "copy":
        hkv, d, bits = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([8, 16])
        layers = rng.choice([1, 1, 2, 4])
        size = 2 * hkv * d * page * bits // 8 * layers
        pages = max(4, min(_log(rng, 16, 8192), int(1.6e9 / size)))
        moves = min(_log(rng, 1, max(2, pages // 3)), int(2.5e8 / size) + 1)
        return {"op": op, "hkv": hkv, "d": d, "page": page, "bits": bits, "layers": layers, "pages": pages, "moves": moves}
    hi = _log(rng, 40, 16384)
    lo = max(1, hi // rng.choice([1, 4, 16]))
    each = (hi + page - 1) // page + 2
    if op == "fork":
        group = rng.choice([2, 3, 4, 8])
        batch = group * _log(rng, 1, 256 // group)
        return {"op": op, "kind": rng.choice(["beams", "prefixes"]), "batch": batch, "group": group, "page": page, "lo": lo,
                "hi": hi, "pages": 2 * batch * each + rng.randrange(100)}
    batch = _log(rng, 1, 256)
    if op == "reserve":
        return {"op": op, "kind": rng.choice(["drafts", "prompts"]), "batch": batch, "page": page, "lo": lo, "hi": hi,
                "pages": batch * each + _log(rng, 1, 4000), "add": rng.randint(1, 8)}
    return {"op": op, "batch": batch, "page": page, "lo": lo, "hi": hi, "pages": batch * each + _log(rng, 1, 4000),
            "gone": rng.choice([2, 3, 5])}


# ------------------------------------------------------------------ inputs
def _spread(i):
    """A fixed ragged sequence in [0, 1)."""
    return (0.381966 + 0.618034 * i + 0.2 * ((i * i) % 5)) % 1.0


def _cuts(case):
    """New tokens of each request: `one` requests have one each, the others share the rest, at least one each."""
    b, t, one = case["batch"], case["tokens"], case["one"]
    if t % b == 0 and not one:
        return [t // b] * b
    many = b - one
    weights = [0.1 + _spread(i) for i in range(many)]
    n = [1 + int((t - b) * w / sum(weights)) for w in weights]
    n[many // 2] += t - one - sum(n)
    out = [1] * b
    for i in range(many):                 # spread between the requests of one token
        out[(i * b) // many] = n[i]
    return out


def _pasts(case):
    """Cached tokens of each request: the most first, the others spread over the range."""
    lo, hi = case["lo"], case["hi"]
    return [hi] + [lo + int((hi + 1 - lo) * _spread(i)) for i in range(1, case["batch"])]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(g, *shape, channels=True):
    """bf16 values of projections: channels of unlike size, as keys have them."""
    x = torch.randn(*shape, generator=g, device="cuda")
    if channels:
        x = x * torch.exp(0.4 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x.bfloat16()


def _pools(s, g, bits, shape):
    """Pools of K and V [..][Hkv][page][d] with, for 8 bits, a power of two for each page and head."""
    s["k_scale"] = s["v_scale"] = None
    flat = (-1,) + tuple(shape[-3:])
    for x in ("k", "v"):
        if bits == 16:
            pool = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        else:
            pool = torch.empty(shape, dtype=E4M3, device="cuda")
            s[x + "_scale"] = torch.ldexp(torch.ones(shape[:-2], device="cuda"),
                                          torch.randint(-8, -5, shape[:-2], generator=g, device="cuda"))
        rows = pool.view(flat)
        step = max(1, 2 ** 27 // (shape[-1] * shape[-2] * shape[-3]))
        for i in range(0, rows.shape[0], step):
            part = torch.randn((min(step, rows.shape[0] - i),) + flat[1:], generator=g, device="cuda")
            rows[i:i + step].copy_(part.bfloat16() if bits == 16 else (part * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3))
        s[x + "_pages"] = pool


def _fill(table, held, order, at, rows):
    """Gives row b of the table `rows[b]` pages of `order` from `at` on, dealt round the requests as they grow."""
    for j in range(max(rows) if rows else 0):
        who = [b for b, n in enumerate(rows) if n > j]
        table[who, j] = order[at:at + len(who)]
        at += len(who)
    held.copy_(torch.tensor(rows, dtype=torch.int32))
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    page = case["page"]
    if case["op"] == "chunk":
        hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["batch"]
        n, past = _cuts(case), _pasts(case)
        total = [x + y for x, y in zip(n, past)]
        need = (max(total) + page - 1) // page
        per = [(x + page - 1) // page for x in total]
        n_pages = sum(per) + 5
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu()
        table, at = torch.full((b, need), -1, dtype=torch.int32), 0
        for i, p in enumerate(per):
            table[i, :p] = order[at:at + p]
            at += p
        s["table"] = table.cuda()
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        s["cu"], s["lens"] = _i32(cu), _i32(total)
        s["max_new"], s["max_len"] = max(n), max(total)
        s["q"] = _normal(g, cu[-1], hq, d, channels=False)
        _pools(s, g, case["bits"], (n_pages, hkv, page, d))
        return s
    n_pages = case["pages"]
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    if case["op"] == "copy":
        _pools(s, g, case["bits"], (case["layers"], n_pages, case["hkv"], page, case["d"]))
        m = case["moves"]
        s["src"], s["dst"] = order[:m].contiguous(), order[m:2 * m].contiguous()
        s["count"] = _i32([m])
        return s
    b, op = case["batch"], case["op"]
    cpu = torch.Generator().manual_seed(seed)
    lens = [case["lo"] + int((case["hi"] + 1 - case["lo"]) * x) for x in torch.rand(b, generator=cpu).tolist()]
    order = order.cpu()
    up = lambda x: (x + page - 1) // page
    width = up(case["hi"] + case.get("add", 0)) + 1
    table, held = torch.full((b, width), -1, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
    parent = list(range(b))
    keep = list(lens)
    if op == "fork":
        k = case["group"]
        if case["kind"] == "beams":       # the beams of a prompt are as long as each other; some go on twice, some end
            for i in range(b):
                keep[i] = lens[i - i % k]
            pick = torch.randint(0, k, (b,), generator=cpu).tolist()
            parent = [i - i % k + pick[i] for i in range(b)]
            lens = keep
        else:                             # the first of each group is a cached prefix, the others become its forks
            for i in range(b):
                base = i - i % k
                if i != base:
                    parent[i] = base
                    keep[i] = max(1, int(lens[base] * (0.5 + 0.5 * _spread(i)))) if i % 2 else lens[base]
        at = _fill(table, held, order, 0, [up(x) for x in lens])
    elif op == "reserve":
        want = [x + case["add"] for x in lens]
        if case["kind"] == "prompts":     # every third request ends; its slot goes to a new prompt of that length
            parent = [-1 if i % 3 == 1 else i for i in range(b)]
            keep = [0 if p < 0 else x for p, x in zip(parent, lens)]
            want = lens
        s["want"] = _i32(want)
        at = _fill(table, held, order, 0, [up(x) for x in keep])
    else:                                 # pages were taken by all requests, and some have ended since
        at = _fill(table, held, order.sort().values, 0, [up(x) for x in lens])
        for i in range(b):
            if i % case["gone"] == 1:
                table[i] = -1
                held[i] = 0
    refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    s["table"], s["held"], s["refs"] = table.cuda(), held.cuda(), refs.cuda()
    s["parent"], s["keep"] = _i32(parent), _i32(keep)
    if op == "compact":
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    return s


# ------------------------------------------------------------------ plain forms
def _plain_chunk(s):
    """All requests padded to the longest, KV head by KV head of scores [batch][r x new][keys]."""
    c = s["case"]
    page, r, hkv, d, b = c["page"], c["hq"] // c["hkv"], c["hkv"], c["d"], c["batch"]
    cu, lens = s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    m, need = s["max_new"], s["table"].shape[1]
    i = torch.arange(m, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                    # [b][m]
    sees = lens[:, None] - new[:, None] + i + 1                                # keys that a token sees
    real = i < new[:, None]
    key = torch.arange(need * page, device="cuda")
    phys = s["table"].long().clamp(min=0)
    o = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], device="cuda")
    q = s["q"].float()

    def rows(x, h):
        pages, scale = s[x + "_pages"], s[x + "_scale"]
        if scale is None:
            return pages[phys, h].float().flatten(1, 2)
        return (pages.view(torch.uint8)[phys, h].view(E4M3).float() * scale[phys, h][..., None, None]).flatten(1, 2)

    hide = key >= sees[..., None]                                              # [b][m][keys]
    for h in range(hkv):
        x = q[at, h * r:(h + 1) * r].transpose(1, 2)                           # [b][r][m][d]
        x = torch.matmul(x, rows("k", h).transpose(1, 2)[:, None]).mul_(1.0 / math.sqrt(d))
        x.masked_fill_(hide[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        v = rows("v", h)
        v = torch.where((key >= lens[:, None])[..., None], torch.zeros_like(v), v)
        y = torch.matmul(x, v[:, None]) / torch.where(total > 0, total, torch.ones_like(total))
        o[at[real], h * r:(h + 1) * r] = y.transpose(1, 2)[real].bfloat16()
        lse[at[real], h * r:(h + 1) * r] = (top + total.log())[..., 0].transpose(1, 2)[real]
    return o, lse


def _plain_copy(s):
    at = torch.arange(s["src"].numel(), device="cuda") < s["count"]
    src, dst = s["src"].long()[at], s["dst"].long()[at]
    for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
        if s[x] is not None:
            pool = s[x].view(torch.uint8) if s[x].dtype == E4M3 else s[x]
            pool[:, dst] = pool[:, src]


def _uses(entries, n):
    return torch.bincount(entries[entries >= 0].long(), minlength=n).to(torch.int32)


def _listed(values, n):
    out = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    out[:values.numel()] = values.to(torch.int32)
    return out


def _plain_fork(s):
    """Request b becomes the first keep[b] tokens of what request parent[b] was (-1: nothing); a page that is filled in
    part belongs to one request: the first of its holders where all hold it so, copies go to the others."""
    table, held, refs, page = s["table"], s["held"], s["refs"], s["case"]["page"]
    b, n = table.shape[0], refs.numel()
    parent, keep = s["parent"].long(), s["keep"].long()
    pages = torch.where(parent >= 0, (keep + page - 1) // page, torch.zeros_like(keep))
    j = torch.arange(table.shape[1], device="cuda")
    new = torch.where(j < pages[:, None], table[parent.clamp(min=0)], torch.full_like(table, -1))
    refs += _uses(new, n) - _uses(table, n)
    row = torch.arange(b, device="cuda")
    partly = (pages > 0) & (keep % page != 0)
    last = new[row, (pages - 1).clamp(min=0)].long().clamp(min=0)
    ones = partly.to(torch.int32)
    holders = torch.zeros(n, dtype=torch.int32, device="cuda").index_add_(0, last, ones)
    first = torch.full((n,), b, dtype=torch.int64, device="cuda").scatter_reduce_(
        0, last, torch.where(partly, row, torch.full_like(row, b)), "amin")
    copy = partly & ~((refs[last] == holders[last]) & (first[last] == row))
    free = (refs == 0).nonzero()[:, 0]
    who = copy.nonzero()[:, 0]
    lost = who[free.numel():]
    who = who[:free.numel()]
    src, dst = last[who], free[:who.numel()]
    refs -= torch.zeros_like(refs).index_add_(0, last, copy.to(torch.int32))
    refs[dst] = 1
    new[who, pages[who] - 1] = dst.to(torch.int32)
    new[lost, pages[lost] - 1] = -1
    pages[lost] -= 1
    table.copy_(new)
    held.copy_(pages)
    return _listed(src, b), _listed(dst, b), _i32([src.numel()])


def _plain_reserve(s):
    """Requests get free pages, the lowest first, in their order, until one asks for more than are left."""
    table, held, refs, page = s["table"], s["held"], s["refs"], s["case"]["page"]
    need = ((s["want"].long() + page - 1) // page - held).clamp(min=0)
    end = need.cumsum(0)
    free = (refs == 0).nonzero()[:, 0]
    given = torch.where(end <= free.numel(), need, torch.zeros_like(need))
    j = torch.arange(table.shape[1], device="cuda")
    mine = (j >= held[:, None]) & (j < (held + given)[:, None])
    rank = (end - need)[:, None] + j - held[:, None]
    pages = free[rank[mine]]
    table[mine] = pages.to(torch.int32)
    refs[pages] = 1
    held += given.to(torch.int32)


def _plain_compact(s):
    """The live pages behind the first `live` places move into the holes before them, both in ascending order."""
    table, refs = s["table"], s["refs"]
    n = refs.numel()
    live = int((refs > 0).sum())
    at = torch.arange(n, device="cuda")
    dst, src = at[(refs == 0) & (at < live)], at[(refs > 0) & (at >= live)]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], table))
    out = refs.clone()
    out[dst] = refs[src]
    out[src] = 0
    s["refs_out"].copy_(out)
    return _listed(src, n // 2), _listed(dst, n // 2), _i32([src.numel()])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from sparse_kv_cache_landmark_gb300 import kvo
        if op == "chunk":
            return kvo.paged_chunk_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], max_new=s["max_new"],
                                        max_len=s["max_len"])
        if op == "copy":
            kvo.paged_copy(s["k_pages"], s["v_pages"], s["src"], s["dst"], s["count"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
        elif op == "fork":
            moves = kvo.paged_fork(s["table"], s["held"], s["refs"], s["parent"], s["keep"], c["page"])
        elif op == "reserve":
            moves = kvo.paged_fork(s["table"], s["held"], s["refs"], s["parent"], s["keep"], c["page"])
            kvo.paged_reserve(s["table"], s["held"], s["refs"], s["want"], c["page"])
        else:
            moves = kvo.paged_compact(s["table"], s["held"], s["refs"], table_out=s["table_out"], refs_out=s["refs_out"])
    else:
        if op == "chunk":
            return _plain_chunk(s)
        if op == "copy":
            _plain_copy(s)
        elif op == "fork":
            moves = _plain_fork(s)
        elif op == "reserve":
            moves = _plain_fork(s)
            _plain_reserve(s)
        else:
            moves = _plain_compact(s)
    if op == "copy":
        return [s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]]
    if op == "compact":
        return [s["table_out"], s["refs_out"], *moves]
    return [s["table"], s["held"], s["refs"], *moves]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    page = case["page"]
    if case["op"] == "chunk":
        hq, hkv, d, w = case["hq"], case["hkv"], case["d"], case["bits"] // 8
        n, past = _cuts(case), _pasts(case)
        keys, t = sum(n) + sum(past), sum(n)
        pages = sum((a + p + page - 1) // page for a, p in zip(n, past))
        pairs = sum(a * (a + 1) // 2 + a * p for a, p in zip(n, past))
        return {"bytes": 2 * w * keys * hkv * d + (8 * pages * hkv if w == 1 else 0) + 4 * pages + 4 * t * hq * d +
                4 * t * hq, "flops": 4 * d * hq * pairs}
    if case["op"] == "copy":
        size = case["hkv"] * (page * case["d"] * case["bits"] // 8 + (4 if case["bits"] == 8 else 0))
        return {"bytes": 2 * 2 * case["layers"] * case["moves"] * size + 8 * case["moves"], "flops": 0}
    b, n = case["batch"], case["pages"]
    each = ((case["lo"] + case["hi"]) // 2 + page - 1) // page
    if case["op"] == "fork":              # old and new entries of the rows that change, and their counts
        rows = b * (case["group"] - 1) // case["group"]
        return {"bytes": 4 * rows * each * 4 + 4 * n, "flops": rows * each}
    if case["op"] == "reserve":           # the pages that change hands, and one look at the counts
        move = b // 3 * each if case["kind"] == "prompts" else b * case["add"] // page + 1
        return {"bytes": 2 * 4 * 2 * move + 4 * n + 16 * b, "flops": move}
    return {"bytes": 2 * 4 * b * ((case["hi"] + page - 1) // page + 1) + 2 * 4 * n, "flops": n}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_chunk(c, s):
    r, page = c["hq"] // c["hkv"], c["page"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n, have = cu[b + 1] - cu[b], lens[b]
        at = s["table"][b, :(have + page - 1) // page].long()
        for g in range(c["hkv"]):
            kv = []
            for x in "kv":
                rows = s[x + "_pages"].view(torch.uint8 if c["bits"] == 8 else torch.bfloat16)[at, g]
                if c["bits"] == 8:
                    rows = rows.view(E4M3).double() * s[x + "_scale"][at, g].double()[:, None, None]
                kv.append(rows.double().flatten(0, 1)[:have])
            k, v = kv
            heads = slice(g * r, (g + 1) * r)
            for i in range(0, n, 512):
                m = min(512, n - i)
                tokens = slice(cu[b] + i, cu[b] + i + m)
                q = s["q"][tokens, heads].double()
                x = torch.einsum("mrd,nd->mrn", q, k) / math.sqrt(c["d"])
                past = torch.arange(have, device="cuda") - (have - n + i)              # key's place behind the first of these
                x.masked_fill_((past > torch.arange(m, device="cuda")[:, None])[:, None, :], -math.inf)
                z = torch.logsumexp(x, dim=-1)
                lse[tokens, heads] = z
                x = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(x - z[..., None]))
                o[tokens, heads] = torch.einsum("mrn,nd->mrd", x, v)
    return o, lse


class _Book:
    """The bookkeeping in plain Python: rows of page ids, and how often each page is named."""

    def __init__(self, s):
        self.rows = [r[:h] for r, h in zip(s["table"].tolist(), s["held"].tolist())]
        self.refs = s["refs"].tolist()
        self.width = s["table"].shape[1]

    def lowest(self):
        return (p for p, n in enumerate(list(self.refs)) if n == 0)

    def fork(self, parent, keep, page):
        old = [list(r) for r in self.rows]
        self.rows = [old[p][:-(-k // page)] if p >= 0 else [] for p, k in zip(parent, keep)]
        for sign, rows in ((-1, old), (1, self.rows)):
            for r in rows:
                for p in r:
                    self.refs[p] += sign
        part = {}
        for b, (r, k) in enumerate(zip(self.rows, keep)):
            if r and k % page:
                part.setdefault(r[-1], []).append(b)
        stays = {p: who[0] for p, who in part.items() if self.refs[p] == len(who)}
        moves, free = [], self.lowest()
        for b in sorted(b for p, who in part.items() for b in who if stays.get(p) != b):
            p, to = self.rows[b].pop(), next(free, None)
            self.refs[p] -= 1
            if to is not None:
                self.refs[to] = 1
                self.rows[b].append(to)
                moves.append((p, to))
        return moves

    def reserve(self, want, page):
        free = list(self.lowest())
        asked = 0
        for r, w in zip(self.rows, want):
            n = max(0, -(-w // page) - len(r))
            if asked + n <= len(free):
                for p in free[asked:asked + n]:
                    r.append(p)
                    self.refs[p] = 1
            asked += n

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        moves = list(zip([p for p in range(live, len(self.refs)) if self.refs[p]], holes))
        to = dict(moves)
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        for a, b in moves:
            self.refs[a], self.refs[b] = 0, self.refs[a]
        return moves

    def table(self):
        return _i32([r + [-1] * (self.width - len(r)) for r in self.rows])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "chunk":
        return _exact_chunk(case, s)
    if op == "copy":
        out = []
        for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
            pool = s[x]
            if pool is not None:
                pool = pool.view(torch.uint8) if pool.dtype == E4M3 else pool.clone()
                for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                    pool[:, b].copy_(pool[:, a])
                pool = pool.view(s[x].dtype) if s[x].dtype == E4M3 else pool
            out.append(pool)
        return out
    book, page = _Book(s), case["page"]
    size = case["batch"] if op != "compact" else case["pages"] // 2
    if op == "compact":
        moves = book.compact()
    else:
        moves = book.fork(s["parent"].tolist(), s["keep"].tolist(), page)
        if op == "reserve":
            book.reserve(s["want"].tolist(), page)
    held = _i32([len(r) for r in book.rows])
    pad = [-1] * (size - len(moves))
    listed_moves = [_i32([a for a, _ in moves] + pad), _i32([b for _, b in moves] + pad), _i32([len(moves)])]
    if op == "compact":
        return [book.table(), _i32(book.refs), *listed_moves]
    return [book.table(), held, _i32(book.refs), *listed_moves]
